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
//
// Measured over the 145 tensors (110 M elements) of a 12-layer model of width 768, fp32
// parameters with bf16 copies: fp32 states and gradients 500 us, 6.6 TB/s, the rate of a copy;
// 8-bit states and bf16 gradients 360 us, 4.9 TB/s (75%): some 50 instructions an element (two
// roots and conversions both ways among them) share the time with the memory.  In a captured graph, with
// the step and the rate on the device, whose powers every block computes first: 32 bits 491 us (host
// scalars 491), 8 bits 363 (353), five small tensors 8.2 (6.2).
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

// The same of two elements.  The packed sum of packed products came out fused (one rounding), so
// the sums are the scalar ones, which never are.
__device__ __forceinline__ float2 sum_of_products(float2 a, float2 b, float2 c, float2 d) {
  const float2 x = mul2(a, b), y = mul2(c, d);
  return make_float2(__fadd_rn(x.x, y.x), __fadd_rn(x.y, y.y));
}

// p - (lr wd p + update): the decay joins the update before the one rounding to p's precision.  As a
// factor 1 - lr wd it would itself be rounded, to a step of 2^-24, the same way in every step and for
// every element (lr wd = 1e-8: no decay at all; 3e-8: twice of it).  An infinite parameter takes the
// decay of the largest number and stays what it is.
__device__ __forceinline__ float decayed(float p) { return fminf(fmaxf(p, -3.402823466e38f), 3.402823466e38f); }

__device__ __forceinline__ float updated(float p, float m, float root, const AdamParams& a, const Factors& f,
                                         float decay) {
  return p - fmaf(decay, decayed(p), f.lr_c1 * m / (root * f.rsqrt_c2 + a.eps));
}

// The same of two elements with the approximate reciprocal (1 unit of 2^-23): the update is a
// small part of the parameter, and a root is at most the root of the largest number.
__device__ __forceinline__ float2 updated2(float2 p, float2 m, float2 root, const AdamParams& a, const Factors& f,
                                           float decay) {
  float2 d = fma2(root, both(f.rsqrt_c2), both(a.eps));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(d.x));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(d.y));
  // p + (-lr wd p - update)
  return add2(p, fma2(make_float2(decayed(p.x), decayed(p.y)), both(-decay), mul2(mul2(m, d), both(-f.lr_c1))));
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
  const float gs = a.grad_scale ? __ldg(a.grad_scale) : 1.f, decay = f.lr * t.weight_decay;
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
      x[e] = updated(x[e], mm[e], sqrtf(vv[e]), a, f, decay);
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

// ------------------------------------------------------------------------ 8-bit states
// A warp takes blocks of 256 elements; lane l holds elements 4 l .. 4 l + 3 and 128 + 4 l ..
// 128 + 4 l + 3 of one, so that every access of the warp is to consecutive bytes.

// largest magnitude over a warp; the integer order of the bits puts infinities above every
// number and NaN above them, so that neither is lost
__device__ __forceinline__ float warp_max_abs(const float2 (&x)[4]) {
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    most = max(most, max(__float_as_uint(x[i].x) & 0x7fffffffu, __float_as_uint(x[i].y) & 0x7fffffffu));
  return __uint_as_float(__reduce_max_sync(0xffffffffu, most));
}

__device__ __forceinline__ uint32_t to_e4m3x2(float2 x) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(x.y), "f"(x.x));
  return r;
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t bits) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)bits));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// the values of a lane's eight codes
__device__ __forceinline__ void decode8(uint2 raw, float scale, float2 (&x)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = mul2(from_e4m3x2((i < 2 ? raw.x : raw.y) >> (16 * (i & 1))), both(scale));
}

__device__ __forceinline__ float block_scale(float most) {
  const float s = __fmul_rn(most, 1.f / 448.f);
  return s < 1.17549435e-38f ? 1.17549435e-38f : s;  // the smallest normal number (NaN stays NaN)
}

// ROOT: a value that is not zero becomes at least the smallest code, 2^-9
template <bool ROOT>
__device__ __forceinline__ uint2 encode8(const float2 (&x)[4], float inv) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 y = mul2(x[i], both(inv));
    if (ROOT) {  // max.NaN: a NaN stays one
      asm("max.NaN.f32 %0, %0, %1;" : "+f"(y.x) : "f"(x[i].x > 0.f ? 0x1p-9f : 0.f));
      asm("max.NaN.f32 %0, %0, %1;" : "+f"(y.y) : "f"(x[i].y > 0.f ? 0x1p-9f : 0.f));
    }
    w[i] = to_e4m3x2(y);
  }
  return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

// A lane's part of one block as loaded.
template <typename P, typename G>
struct Loaded8 {
  Raw8<P> p;
  Raw8<G> g;
  uint2 m, v;
  float m_scale, v_scale;
  __device__ __forceinline__ void load(const AdamTensor& t, long long block, int lane) {
    const long long at = block * kAdamBlock;
    p.template load<true>(static_cast<const P*>(t.p) + at, lane, 32);
    g.template load<true>(static_cast<const G*>(t.g) + at, lane, 32);
    const uint32_t* mm = reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(t.m) + at);
    const uint32_t* vv = reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(t.v) + at);
    m = make_uint2(__ldcs(mm + lane), __ldcs(mm + 32 + lane));
    v = make_uint2(__ldcs(vv + lane), __ldcs(vv + 32 + lane));
    m_scale = t.m_scale[block];
    v_scale = t.v_scale[block];
  }
  // the last block of a tensor, of which `rest` elements exist; the others become zero
  __device__ __forceinline__ void load_part(const AdamTensor& t, long long block, int lane, int rest) {
    const long long at = block * kAdamBlock;
    float x[8], y[8];
    m = v = make_uint2(0, 0);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = share<true>(e, lane, 32);
      x[e] = i < rest ? load1(static_cast<const P*>(t.p) + at + i) : 0.f;
      y[e] = i < rest ? load1(static_cast<const G*>(t.g) + at + i) : 0.f;
      const uint32_t mc = i < rest ? static_cast<const uint8_t*>(t.m)[at + i] : 0;
      const uint32_t vc = i < rest ? static_cast<const uint8_t*>(t.v)[at + i] : 0;
      (e < 4 ? m.x : m.y) |= mc << (8 * (e & 3));
      (e < 4 ? v.x : v.y) |= vc << (8 * (e & 3));
    }
    p.put(x);
    g.put(y);
    m_scale = t.m_scale[block];
    v_scale = t.v_scale[block];
  }
};

struct Stepped8 {
  float2 x[4];
  uint2 m, v;
  float m_scale, v_scale;
};

// The step of one block.  `rest`: elements that exist (the others must not poison the scales:
// zero times a scale that is NaN is not zero).
template <bool PART, typename P, typename G>
__device__ __forceinline__ Stepped8 step8(const Loaded8<P, G>& in, const AdamParams& a, const Factors& f, float gs,
                                          float decay, int lane, int rest) {
  Stepped8 out;
  float2 m[4], r[4];
  decode8(in.m, in.m_scale, m);
  decode8(in.v, in.v_scale, r);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 g = mul2(in.g.get(i), both(gs));
    m[i] = sum_of_products(m[i], both(a.b1), g, both(a.r1));
    const float2 v = sum_of_products(mul2(r[i], r[i]), both(a.b2), mul2(g, g), both(a.r2));
    r[i] = make_float2(sqrtf(v.x), sqrtf(v.y));
    out.x[i] = updated2(in.p.get(i), m[i], r[i], a, f, decay);
    if (PART) {
      const int e = share<true>(2 * i, lane, 32);
      if (e >= rest) m[i].x = r[i].x = 0.f;
      if (e + 1 >= rest) m[i].y = r[i].y = 0.f;
    }
  }
  out.m_scale = block_scale(warp_max_abs(m));
  out.v_scale = block_scale(warp_max_abs(r));
  out.m = encode8<false>(m, 1.f / out.m_scale);
  out.v = encode8<true>(r, 1.f / out.v_scale);
  return out;
}

template <typename P, typename G, int N>
__global__ void __launch_bounds__(kAdamThreads) adamw8_kernel(const __grid_constant__ AdamTable<N> table, int count,
                                                              AdamParams a) {
  const AdamTensor& t = find_tensor(table, count);
  const Factors f = step_factors(a);
  const float gs = a.grad_scale ? __ldg(a.grad_scale) : 1.f, decay = f.lr * t.weight_decay;
  const int lane = threadIdx.x % 32, warps = kAdamThreads / 32;
  const int per = a.chunk / kAdamBlock;
  const long long first = (long long)(blockIdx.x - t.first_block) * per;
  const long long full = t.n / kAdamBlock, last = first + per < full ? first + per : full;  // whole blocks
  P* p = static_cast<P*>(t.p);
  __nv_bfloat16* copy = static_cast<__nv_bfloat16*>(t.copy);
  long long b = first + threadIdx.x / 32;
  Loaded8<P, G> cur, next;
  if (b < last) next.load(t, b, lane);
  for (; b < last; b += warps) {
    cur = next;
    if (b + warps < last) next.load(t, b + warps, lane);
    const Stepped8 s = step8<false>(cur, a, f, gs, decay, lane, kAdamBlock);
    const long long at = b * kAdamBlock;
    store_shared8<true>(p + at, lane, 32, kAdamBlock, s.x);
    if (copy) store_shared8<true>(copy + at, lane, 32, kAdamBlock, s.x);
    uint32_t* mm = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(t.m) + at);
    uint32_t* vv = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(t.v) + at);
    mm[lane] = s.m.x;
    mm[32 + lane] = s.m.y;
    vv[lane] = s.v.x;
    vv[32 + lane] = s.v.y;
    if (lane == 0) {
      t.m_scale[b] = s.m_scale;
      t.v_scale[b] = s.v_scale;
    }
  }
  // b is now the first of this warp's blocks behind the whole ones of the chunk: the part at the
  // tensor's end belongs to the warp that would have had it
  const int rest = (int)(t.n - full * kAdamBlock);
  if (b != full || rest == 0 || full >= first + per) return;
  cur.load_part(t, full, lane, rest);
  const Stepped8 s = step8<true>(cur, a, f, gs, decay, lane, rest);
  const long long at = full * kAdamBlock;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int i = share<true>(e, lane, 32);
    if (i >= rest) continue;
    const float x = e & 1 ? s.x[e / 2].y : s.x[e / 2].x;
    st1<P>(p + at + i, x);
    if (copy) st1<__nv_bfloat16>(copy + at + i, x);
    static_cast<uint8_t*>(t.m)[at + i] = (uint8_t)((e < 4 ? s.m.x : s.m.y) >> (8 * (e & 3)));
    static_cast<uint8_t*>(t.v)[at + i] = (uint8_t)((e < 4 ? s.v.x : s.v.y) >> (8 * (e & 3)));
  }
  if (lane == 0) {
    t.m_scale[full] = s.m_scale;
    t.v_scale[full] = s.v_scale;
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
