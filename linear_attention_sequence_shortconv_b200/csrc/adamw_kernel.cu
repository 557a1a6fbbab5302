// One AdamW step over many tensors in one launch.
//
//   g = grad_scale * grad;  m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2
//   p = p (1 - lr wd) - (lr / c1) m / (sqrt(v) / sqrt(c2) + eps),  c1 = 1 - b1^step, c2 = 1 - b2^step
//
// States in 32 bits, or in 8: blocks of 256 consecutive elements hold m, and the root of v, as
// e4m3 times one fp32 scale, the block's largest magnitude / 448.  The root is held rather
// than v because it spans half the exponents; a root that is not zero is never held as zero
// (its update would have only eps below it).  The parameter's update takes the new moments
// before they are rounded to 8 bits.
//
// Bound by memory: 28 bytes an element in fp32 (16 with 8-bit states and fp32 gradients).  The
// tensors' descriptors are a kernel parameter, so that the step needs no copy to the device
// and a captured graph holds them; a block finds its tensor by bisection.
#include "adamw.cuh"
#include "rowops.cuh"

namespace prism {

namespace {

constexpr int kAdamThreads = 256;

template <int N>
struct AdamTable {
  AdamTensor t[N];
};

// fp32 scalars of the step
struct Factors {
  float lr, lr_c1, rsqrt_c2;
};

// The learning rate and the bias corrections, in fp64, where the step or the rate is read
// from the device; the host has computed them otherwise.
__device__ __forceinline__ Factors step_factors(const AdamParams& p) {
  Factors f{p.lr, p.lr_c1, p.rsqrt_c2};
  if (p.step_dev || p.lr_dev) {
    __shared__ Factors shared;
    if (threadIdx.x == 0) {
      const int step = p.step_dev ? max(1, *p.step_dev) : p.step;
      const double lr = p.lr_dev ? (double)*p.lr_dev : p.lr64;
      shared.lr = (float)lr;
      shared.lr_c1 = (float)(lr / (1.0 - pow(p.beta1, (double)step)));
      shared.rsqrt_c2 = (float)(1.0 / sqrt(1.0 - pow(p.beta2, (double)step)));
    }
    __syncthreads();
    f = shared;
  }
  return f;
}

// Products and sums of the moments are rounded one by one (no fused multiply-add), so that a
// moment, and what 8 bits hold of it, is the same as in separate fp32 operations.
__device__ __forceinline__ float moment(float m, float x, float b, float rest) {
  return __fadd_rn(__fmul_rn(m, b), __fmul_rn(x, rest));
}

__device__ __forceinline__ float updated(float p, float m, float root, const AdamParams& a, const Factors& f,
                                         float keep) {
  return p * keep - f.lr_c1 * m / (root * f.rsqrt_c2 + a.eps);
}

template <int N>
__device__ __forceinline__ const AdamTensor& find_tensor(const AdamTable<N>& table, int count) {
  int lo = 0, hi = count - 1;  // the last tensor whose first block is not behind this one
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (table.t[mid].first_block <= blockIdx.x) lo = mid;
    else hi = mid - 1;
  }
  return table.t[lo];
}

template <typename P, typename G, int N>
__global__ void __launch_bounds__(kAdamThreads) adamw32_kernel(const __grid_constant__ AdamTable<N> table, int count,
                                                               AdamParams a) {
  const AdamTensor& t = find_tensor(table, count);
  const Factors f = step_factors(a);
  const float gs = a.grad_scale ? __ldg(a.grad_scale) : 1.f, keep = 1.f - f.lr * t.weight_decay;
  const long long first = (long long)(blockIdx.x - t.first_block) * kAdamChunk;
  P* p = static_cast<P*>(t.p);
  const G* g = static_cast<const G*>(t.g);
  float* m = static_cast<float*>(t.m);
  float* v = static_cast<float*>(t.v);
  __nv_bfloat16* copy = static_cast<__nv_bfloat16*>(t.copy);
#pragma unroll
  for (int it = 0; it < kAdamChunk / (8 * kAdamThreads); ++it) {
    const long long i = first + (long long)(it * kAdamThreads + threadIdx.x) * 8;
    if (i >= t.n) break;
    const int rest = t.n - i < 8 ? (int)(t.n - i) : 8;
    float x[8], y[8], mm[8], vv[8];
    if (rest == 8) {
      load8(p + i, x);
      load8(g + i, y);
      load8(m + i, mm);
      load8(v + i, vv);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] = e < rest ? load1(p + i + e) : 0.f;
        y[e] = e < rest ? load1(g + i + e) : 0.f;
        mm[e] = e < rest ? m[i + e] : 0.f;
        vv[e] = e < rest ? v[i + e] : 0.f;
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float gr = y[e] * gs;
      mm[e] = moment(mm[e], gr, a.b1, a.r1);
      vv[e] = moment(vv[e], __fmul_rn(gr, gr), a.b2, a.r2);
      x[e] = updated(x[e], mm[e], sqrtf(vv[e]), a, f, keep);
    }
    if (rest == 8) {
      store8(p + i, x);
      store8(m + i, mm);
      store8(v + i, vv);
      if (copy) store8(copy + i, x);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (e >= rest) break;
        st1<P>(p + i + e, x[e]);
        m[i + e] = mm[e];
        v[i + e] = vv[e];
        if (copy) st1<__nv_bfloat16>(copy + i + e, x[e]);
      }
    }
  }
}

// largest magnitude over a warp; the integer order of the bits puts infinities above every
// number and NaN above them, so that neither is lost
__device__ __forceinline__ float warp_max_abs(const float (&x)[8]) {
  uint32_t most = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) most = max(most, __float_as_uint(x[e]) & 0x7fffffffu);
  return __uint_as_float(__reduce_max_sync(0xffffffffu, most));
}

__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void from_e4m3x2(uint32_t bits, float& lo, float& hi) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)bits));
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  lo = f.x;
  hi = f.y;
}

__device__ __forceinline__ void decode8(uint2 raw, float scale, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    from_e4m3x2(((i < 2 ? raw.x : raw.y) >> (16 * (i & 1))) & 0xffffu, lo, hi);
    x[2 * i] = __fmul_rn(lo, scale);
    x[2 * i + 1] = __fmul_rn(hi, scale);
  }
}

__device__ __forceinline__ float block_scale(float most) {
  const float s = __fmul_rn(most, 1.f / 448.f);
  return s < 1.17549435e-38f ? 1.17549435e-38f : s;  // the smallest normal number (NaN stays NaN)
}

__device__ __forceinline__ uint2 encode8(const float (&x)[8], float inv) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = to_e4m3x2(__fmul_rn(x[2 * i], inv), __fmul_rn(x[2 * i + 1], inv));
  return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

// One warp per block of 256 elements, eight per lane.
template <typename P, typename G, int N>
__global__ void __launch_bounds__(kAdamThreads) adamw8_kernel(const __grid_constant__ AdamTable<N> table, int count,
                                                              AdamParams a) {
  const AdamTensor& t = find_tensor(table, count);
  const Factors f = step_factors(a);
  const float gs = a.grad_scale ? __ldg(a.grad_scale) : 1.f, keep = 1.f - f.lr * t.weight_decay;
  const long long first = (long long)(blockIdx.x - t.first_block) * kAdamChunk;
  P* p = static_cast<P*>(t.p);
  const G* g = static_cast<const G*>(t.g);
  uint8_t* m = static_cast<uint8_t*>(t.m);
  uint8_t* v = static_cast<uint8_t*>(t.v);
  __nv_bfloat16* copy = static_cast<__nv_bfloat16*>(t.copy);
#pragma unroll
  for (int it = 0; it < kAdamChunk / (8 * kAdamThreads); ++it) {
    const long long i = first + (long long)(it * kAdamThreads + threadIdx.x) * 8;
    const long long block = i / kAdamBlock;  // the same for the whole warp
    if (block * kAdamBlock >= t.n) break;
    const int rest = t.n - i >= 8 ? 8 : t.n > i ? (int)(t.n - i) : 0;
    float x[8], y[8], mm[8], rr[8];
    const float ms = t.m_scale[block], vs = t.v_scale[block];
    if (rest == 8) {
      load8(p + i, x);
      load8(g + i, y);
      decode8(__ldcs(reinterpret_cast<const uint2*>(m + i)), ms, mm);
      decode8(__ldcs(reinterpret_cast<const uint2*>(v + i)), vs, rr);
    } else {
      uint32_t mb[2] = {0, 0}, vb[2] = {0, 0};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] = e < rest ? load1(p + i + e) : 0.f;
        y[e] = e < rest ? load1(g + i + e) : 0.f;
        if (e < rest) {
          mb[e / 4] |= (uint32_t)m[i + e] << (8 * (e & 3));
          vb[e / 4] |= (uint32_t)v[i + e] << (8 * (e & 3));
        }
      }
      decode8(make_uint2(mb[0], mb[1]), ms, mm);
      decode8(make_uint2(vb[0], vb[1]), vs, rr);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float gr = __fmul_rn(y[e], gs);
      mm[e] = moment(mm[e], gr, a.b1, a.r1);
      rr[e] = sqrtf(moment(__fmul_rn(rr[e], rr[e]), __fmul_rn(gr, gr), a.b2, a.r2));
      x[e] = updated(x[e], mm[e], rr[e], a, f, keep);
      if (e >= rest) mm[e] = rr[e] = 0.f;  // behind the tensor's end (0 * NaN of a poisoned scale)
    }
    const float ms_new = block_scale(warp_max_abs(mm)), vs_new = block_scale(warp_max_abs(rr));
    const uint2 mc = encode8(mm, 1.f / ms_new);
    uint2 vc = encode8(rr, 1.f / vs_new);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      uint32_t& word = e < 4 ? vc.x : vc.y;
      if (rr[e] > 0.f && ((word >> (8 * (e & 3))) & 0xffu) == 0) word |= 1u << (8 * (e & 3));
    }
    if (rest == 8) {
      store8(p + i, x);
      *reinterpret_cast<uint2*>(m + i) = mc;
      *reinterpret_cast<uint2*>(v + i) = vc;
      if (copy) store8(copy + i, x);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (e >= rest) break;
        st1<P>(p + i + e, x[e]);
        m[i + e] = (uint8_t)((e < 4 ? mc.x : mc.y) >> (8 * (e & 3)));
        v[i + e] = (uint8_t)((e < 4 ? vc.x : vc.y) >> (8 * (e & 3)));
        if (copy) st1<__nv_bfloat16>(copy + i + e, x[e]);
      }
    }
    if (threadIdx.x % 32 == 0) {
      t.m_scale[block] = ms_new;
      t.v_scale[block] = vs_new;
    }
  }
}

template <typename P, typename G, int N>
void adamw_launch_n(const AdamTensor* tensors, int count, unsigned blocks, const AdamParams& a, int bits,
                    cudaStream_t stream) {
  AdamTable<N> table;
  for (int i = 0; i < count; ++i) table.t[i] = tensors[i];
  for (int i = count; i < N; ++i) table.t[i] = AdamTensor{};
  if (bits == 32)
    adamw32_kernel<P, G, N><<<blocks, kAdamThreads, 0, stream>>>(table, count, a);
  else
    adamw8_kernel<P, G, N><<<blocks, kAdamThreads, 0, stream>>>(table, count, a);
}

template <typename P, typename G>
cudaError_t adamw_launch(const AdamTensor* tensors, int count, unsigned blocks, const AdamParams& a, int bits,
                         cudaStream_t stream) {
  if (count <= 8) adamw_launch_n<P, G, 8>(tensors, count, blocks, a, bits, stream);
  else if (count <= 48) adamw_launch_n<P, G, 48>(tensors, count, blocks, a, bits, stream);
  else adamw_launch_n<P, G, kAdamMostTensors>(tensors, count, blocks, a, bits, stream);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_adamw(const AdamTensor* tensors, int count, unsigned blocks, const AdamParams& a, int p_dtype,
                         int g_dtype, int bits, cudaStream_t stream) {
  if (p_dtype == PRISM_FP32)
    return g_dtype == PRISM_FP32 ? adamw_launch<float, float>(tensors, count, blocks, a, bits, stream)
                                 : adamw_launch<float, __nv_bfloat16>(tensors, count, blocks, a, bits, stream);
  return g_dtype == PRISM_FP32 ? adamw_launch<__nv_bfloat16, float>(tensors, count, blocks, a, bits, stream)
                               : adamw_launch<__nv_bfloat16, __nv_bfloat16>(tensors, count, blocks, a, bits, stream);
}

}  // namespace prism
