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

// Two fp32 operations in one instruction (sm_100a's packed forms): these kernels issue several
// operations per loaded byte, so that their rate would be the limit otherwise.
__device__ __forceinline__ unsigned long long bits2(float2 a) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
  return r;
}
__device__ __forceinline__ float2 float2_of(unsigned long long r) {
  float2 a;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(r));
  return a;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
  return float2_of(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
  return float2_of(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
  return float2_of(r);
}
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }
__device__ __forceinline__ float2 unpack_bf16(uint32_t w) {  // a bf16 is the upper half of the fp32 of the same value
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// How W neighbouring threads share 8 W consecutive elements.  Thread l holds eight: in 16-bit
// rows elements 8 l .. 8 l + 7 (16 bytes), else 4 l .. 4 l + 3 and 4 W + 4 l .. 4 W + 4 l + 3, so
// that every access of the threads is to consecutive bytes (a thread that took the two halves
// of a 32-byte sector in turn would have it moved twice).
template <bool WIDE>  // WIDE: fp32 rows among them
__device__ __forceinline__ int share(int e, int l, int W) {
  return WIDE ? e / 4 * 4 * W + 4 * l + e % 4 : 8 * l + e;
}

// Eight elements of a thread as loaded, and as pairs of fp32 numbers.
template <typename T>
struct Raw8 {
  static constexpr int kPieces = (int)sizeof(T) / 2;  // of 16 bytes
  uint4 v[kPieces];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int h = 0; h < kPieces; ++h) v[h] = make_uint4(0, 0, 0, 0);
  }
  // row: the first of the 8 W elements
  template <bool WIDE>
  __device__ __forceinline__ void load(const T* row, int l, int W) {
    if (sizeof(T) == 2 && WIDE) {
      const uint2 a = __ldcs(reinterpret_cast<const uint2*>(row + share<true>(0, l, W)));
      const uint2 b = __ldcs(reinterpret_cast<const uint2*>(row + share<true>(4, l, W)));
      v[0] = make_uint4(a.x, a.y, b.x, b.y);
    } else {
#pragma unroll
      for (int h = 0; h < kPieces; ++h) v[h] = __ldcs(reinterpret_cast<const uint4*>(row + share<WIDE>(4 * h, l, W)));
    }
  }
  // from fp32 values (exact where they came from a T)
  __device__ __forceinline__ void put(const float (&x)[8]) {
    if (sizeof(T) == 2) {
      v[0] = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
    } else {
#pragma unroll
      for (int h = 0; h < kPieces; ++h)
        v[h] = make_uint4(__float_as_uint(x[4 * h % 8]), __float_as_uint(x[(4 * h + 1) % 8]),
                          __float_as_uint(x[(4 * h + 2) % 8]), __float_as_uint(x[(4 * h + 3) % 8]));
    }
  }
  __device__ __forceinline__ float2 get(int i) const {  // i: a constant after unrolling
    const uint4 q = v[sizeof(T) == 4 ? i / 2 % kPieces : 0];
    if (sizeof(T) == 4)
      return i & 1 ? make_float2(__uint_as_float(q.z), __uint_as_float(q.w))
                   : make_float2(__uint_as_float(q.x), __uint_as_float(q.y));
    return unpack_bf16(i == 0 ? q.x : i == 1 ? q.y : i == 2 ? q.z : q.w);
  }
};

// Eight elements of a thread into row[0 .. 8 W), of which the first n exist.
template <bool WIDE>
__device__ __forceinline__ void store_shared8(float* row, int l, int W, int n, const float2 (&x)[4]) {
  static_assert(WIDE, "fp32 rows");
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int e = share<true>(4 * h, l, W);
    if (e < n) *reinterpret_cast<float4*>(row + e) = make_float4(x[2 * h].x, x[2 * h].y, x[2 * h + 1].x, x[2 * h + 1].y);
  }
}
template <bool WIDE>
__device__ __forceinline__ void store_shared8(__nv_bfloat16* row, int l, int W, int n, const float2 (&x)[4]) {
  const uint4 v = make_uint4(pack_bf16(x[0].x, x[0].y), pack_bf16(x[1].x, x[1].y), pack_bf16(x[2].x, x[2].y),
                             pack_bf16(x[3].x, x[3].y));
  if (WIDE) {
    const int a = share<true>(0, l, W), b = share<true>(4, l, W);
    if (a < n) *reinterpret_cast<uint2*>(row + a) = make_uint2(v.x, v.y);
    if (b < n) *reinterpret_cast<uint2*>(row + b) = make_uint2(v.z, v.w);
  } else if (8 * l < n) {
    *reinterpret_cast<uint4*>(row + 8 * l) = v;
  }
}

// A ring of `STAGES` sets of N 16-byte pieces in shared memory, private to a thread: the thread
// copies what it will read itself (asynchronously), so that the copies of the next STAGES - 1
// sets are in flight without registers and no thread waits for another.  A set is filled again
// only after the thread has used the values that it read from it.
template <int N, int STAGES>
struct Ring {
  uint4* base;  // this thread's first slot; consecutive threads have consecutive slots
  int threads, stage;
  __device__ __forceinline__ Ring(void* smem)
      : base(static_cast<uint4*>(smem) + threadIdx.x), threads(blockDim.x), stage(0) {}
  static __host__ __device__ constexpr size_t bytes(int threads) { return (size_t)STAGES * N * 16 * threads; }
  // Eight of the elements row[0 .. 8 W) into the pieces from `at` on of the set that lies `ahead`
  // sets behind the next one to be read.  Only the first n elements of the row exist; the
  // others become zero, and `any` (readable) stands for their address.
  template <bool WIDE, typename T>
  __device__ __forceinline__ void copy(int ahead, int at, const T* row, int l, int W, int n, const void* any) {
    int s = stage + ahead;
    s = s >= STAGES ? s - STAGES : s;
    const uint32_t dst = (uint32_t)__cvta_generic_to_shared(base + (s * N + at) * threads);
#pragma unroll
    for (int h = 0; h < (WIDE ? 2 : 1); ++h) {
      const int e = share<WIDE>(4 * h, l, W);
      const bool ok = e < n;
      const void* src = ok ? row + e : any;
      if (sizeof(T) == 2 && WIDE)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst + 8 * h), "l"(src), "r"(ok ? 8 : 0)
                     : "memory");
      else
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + 16 * h * threads), "l"(src),
                     "r"(ok ? 16 : 0) : "memory");
    }
  }
  __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
  // the next set is complete (one commit per set, in order)
  __device__ __forceinline__ void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory"); }
  __device__ __forceinline__ void drain() { asm volatile("cp.async.wait_all;" ::: "memory"); }
  template <typename T>
  __device__ __forceinline__ Raw8<T> read(int at) const {
    Raw8<T> r;
#pragma unroll
    for (int h = 0; h < Raw8<T>::kPieces; ++h) r.v[h] = base[(stage * N + at + h) * threads];
    return r;
  }
  __device__ __forceinline__ void advance() { stage = stage + 1 == STAGES ? 0 : stage + 1; }
};

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
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return div32(n); }
};

// Whether token n = b T + t of a right-padded batch is a valid step (t < lengths[b]).
template <typename Index>
__device__ __forceinline__ bool token_valid(Index n, const FastDiv& T, const int32_t* lengths) {
  if (!lengths) return true;
  const Index b = T.div(n);
  return (long long)(n - b * T.d) < __ldg(lengths + b);
}

// Programmatic launch of the next kernel of a chain: it may start once every block of this one
// has said so, and waits for this one's end before it reads its results.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// A launch that may overlap the end of the one before it (whose results its kernel waits for).
template <typename... Args>
cudaError_t launch_chained(void (*kernel)(Args...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                           Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
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
  float* d_weight;
  long long rows, gate_stride;
  FastDiv T, H;
  float eps;
  bool by_token;  // rows are found by their tokens: a strided gate, or lengths
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
  float* part;         // backward: [blocks, nvec, D] column sums of the vectors' gradients
  float* sums[3];      // the gradients of weight, then of post_weight and scale as far as given
  long long rows;
  FastDiv T;
  int D, tpr, groups;
  float res_scale, eps, inv_D;
};

}  // namespace prism
