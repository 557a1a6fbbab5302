// Descriptors of the AdamW step's tensors and scalars.
#pragma once

#include <stdint.h>

namespace prism {

constexpr int kAdamBlock = 256;         // elements under one scale of the 8-bit states
constexpr int kAdamChunk = 4096;        // elements of one thread block (a multiple of kAdamBlock)
constexpr int kAdamMostTensors = 440;   // of one launch: 440 * 72 bytes of the 32764 for parameters

struct AdamTensor {
  void* p;
  const void* g;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  void* copy;
  long long n;
  float weight_decay;
  unsigned first_block;
};

struct AdamParams {
  const float* grad_scale;  // device scalars, or NULL
  const int32_t* step_dev;
  const float* lr_dev;
  double lr64, beta1, beta2;
  int step;
  float lr, lr_c1, rsqrt_c2;  // what the host computed (unused with step_dev or lr_dev)
  float b1, r1, b2, r2, eps;  // betas and 1 - betas
};

}  // namespace prism
