// Helpers of the row-wise kernels (norms, embedding): eight consecutive elements per thread
// as 16-byte accesses, row validity of right-padded batches, and the reduction of per-block
// column sums.
#pragma once

#include "common.cuh"

namespace prism {

constexpr int kSMs = 148;  // B200

// Eight consecutive elements at p (16-byte aligned).  Read once by the kernels that call
// this, and possibly rewritten in place by the same thread, so a coherent streaming load.
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
  const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 raw = __ldcs(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // a bf16 is the upper half of the fp32 of the same value
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}
// one element, coherent (load8's scalar form)
__device__ __forceinline__ float load1(const float* p) { return __ldcs(p); }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) {
  return __uint_as_float((uint32_t)__ldcs(reinterpret_cast<const unsigned short*>(p)) << 16);
}
__device__ __forceinline__ void zero8(float (&x)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = 0.f;
}

// Division by an invariant integer 1 <= d < 2^31 as a multiplication (Granlund and Montgomery,
// "Division by Invariant Integers using Multiplication", 1994, figure 4.1): with
// l = ceil(log2 d) and m = floor(2^32 (2^l - d) / d) + 1, n / d = (t + (n - t) / 2) / 2^(l - 1)
// where t = m n / 2^32.  Dividends of 2^32 and more take the plain division.
struct FastDiv {
  uint32_t d, mul, shift;
  FastDiv() : d(1), mul(1), shift(0) {}
  explicit FastDiv(int divisor) : d((uint32_t)divisor), shift(0) {
    while ((1ull << shift) < d) ++shift;
    mul = (uint32_t)(((1ull << 32) * ((1ull << shift) - d)) / d + 1);
  }
  __device__ __forceinline__ uint32_t div32(uint32_t n) const {
    const uint32_t t = __umulhi(mul, n);
    return shift ? (t + ((n - t) >> 1)) >> (shift - 1) : n;
  }
  __device__ __forceinline__ long long div(long long n) const {
    return n >> 32 ? n / d : (long long)div32((uint32_t)n);
  }
};

// Whether token n = b T + t of a right-padded batch is a valid step (t < lengths[b]).
__device__ __forceinline__ bool token_valid(long long n, const FastDiv& T, const int32_t* lengths) {
  if (!lengths) return true;
  const long long b = T.div(n);
  return n - b * T.d < __ldg(lengths + b);
}

// out[v][c] = sum over blocks of part[block][v][c], v < 3 vectors of width D, in a fixed order.
struct ColumnSumParams {
  const float* part;  // [blocks, nvec, D]
  float* out[3];
  int blocks, nvec, D;
};
cudaError_t launch_column_sum(const ColumnSumParams& p, cudaStream_t stream);

// Pointers and sizes of one gated norm call, forward or backward (device pointers).
struct GatedNormParams {
  const void* o;
  const void* gate;
  const float* weight;
  const void* dy;
  const int32_t* lengths;
  void* y;       // forward: y; backward: d_o
  void* d_gate;
  float* part;   // backward: [blocks, d] column sums
  long long rows, gate_stride;
  FastDiv T, H;
  float eps;
};

// Pointers and sizes of one block norm call, forward or backward (device pointers).
struct BlockNormParams {
  const void* x;       // forward: x; backward: the stored x'
  const void* y;
  const float* post_weight;
  const float* scale;
  const float* weight;
  const void* dh;
  const void* dx_in;
  const int32_t* lengths;
  void* x_out;         // forward: x'; backward: dx
  void* h;             // forward: h; backward: dy
  float* part;         // backward: [blocks, nvec, D] column sums (weight, then post_weight, then scale)
  long long rows;
  FastDiv T;
  int D, tpr, groups;
  float res_scale, eps;
};

}  // namespace prism
