// Descriptors of the AdamW step's tensors and scalars.
#pragma once

#include <stdint.h>

namespace prism {

constexpr int kAdamBlock = 256;         // elements under one scale of the 8-bit states
constexpr int kAdamChunk = 4096;        // least elements of one thread block (a multiple of kAdamBlock)
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

// Elements of a thread block.  8-bit states: longer chunks where they still give every SM several
// blocks, since a warp then fetches one block of states while it works on another.
inline int adam_chunk(long long elements, int bits) {
  int chunk = kAdamChunk;
  while (bits == 8 && chunk < 4 * kAdamChunk && elements / chunk > 16 * 148) chunk *= 2;
  return chunk;
}

struct AdamParams {
  const float* grad_scale;  // device scalars, or NULL
  const int32_t* step_dev;
  const float* lr_dev;
  double lr64, beta1, beta2;
  int step;
  float lr, lr_c1, rsqrt_c2;  // what the host computed (unused with step_dev or lr_dev)
  float b1, r1, b2, r2, eps;  // betas and 1 - betas
  int chunk;                  // elements of a thread block (8-bit states)
};

}  // namespace prism
