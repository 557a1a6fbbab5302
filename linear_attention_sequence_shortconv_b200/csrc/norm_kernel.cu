// The norms around the mixer, forward and backward.
//
// gated norm, one row per (token, head) of the mixer's readout o (width d = d_v):
//   r = 1 / sqrt(mean(o^2) + eps),  xh = o r,  y = xh w act(g)
//   backward of dy:  dg = dy xh w act'(g);  dw = sum_rows dy act(g) xh;
//                    t = dy act(g) w;  do = r (t - xh mean(t xh))
//
// block norm, one row per token of the residual stream x (width D), y the block's output:
//   z = y, or y ry wp with ry = 1 / sqrt(mean(y^2) + eps);  x' = x + k z, k = res_scale scale
//   r = 1 / sqrt(mean(x'^2) + eps),  h = x' r w
//   backward of dh and dx', from the stored x':  t = dh w,  xh = x' r
//     dx = dx' + r (t - xh mean(t xh));  dw = sum_rows dh xh;  dscale = res_scale sum_rows dx z
//     dz = k dx;  dwp = sum_rows dz yh, yh = y ry;  u = dz wp;  dy = ry (u - yh mean(u yh))
//
// All of it is a few operations per byte: the kernels are bound by memory.  Every tensor is
// read once and written once; statistics are recomputed in the backward, since its rows pass
// through registers anyway.  Rows of padding (t >= lengths[b]) are not read: their outputs
// are zero and they add nothing to the weights' gradients.
//
// Measured on a B200 in a loop over three sets of tensors, with the share of the copy rate of
// 6.56 TB/s: gated norm, 130M-LM layer (B 16, T 2048, H 6, d 128, bf16, strided gate) forward
// 29 us, 78%; recommendation layer (B 128, T 1024, H 2, d 64, ragged) backward 27 us, 72%;
// block norm, 130M LM (B 16, T 2048, D 768) forward with an fp32 stream 58 us, 80%, backward in
// bf16 59 us, 78%.  What was in the way before the memory: the instructions (half of what is
// left are conversions, sums and exponentials, in packed pairs where the hardware has them),
// and 32-byte sectors moved in two halves.
#include <type_traits>

#include "rowops.cuh"

namespace prism {

// Blocks of the persistent kernels; the backward ones set the number of partial column sums.
int gated_norm_bwd_blocks(long long rows, int d) {
  const long long per = 256 / (d / 8), need = (rows + per - 1) / per;
  return (int)(need < 4 * kSMs ? need : 4 * kSMs);
}
int block_norm_blocks(long long rows, int D, bool bwd, int x_bytes, int bytes);

namespace {

enum { kGateNone = 0, kGateSilu = 1, kGateSigmoid = 2 };

// 1 / (1 + e^-g) of two gates.  fp32 outputs take the accurate exponential and division; for
// bf16 outputs the approximate instructions' error (a few units of 2^-23 of the exponent's
// argument) is far below the rounding to 8 bits.
template <typename T>
__device__ __forceinline__ float2 sigmoid2(float2 g);
template <>
__device__ __forceinline__ float2 sigmoid2<float>(float2 g) {
  return make_float2(1.f / (1.f + expf(-g.x)), 1.f / (1.f + expf(-g.y)));
}
template <>
__device__ __forceinline__ float2 sigmoid2<__nv_bfloat16>(float2 g) {
  float2 e = mul2(g, both(-1.4426950408889634f));  // log2(e)
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.x));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.y));
  e = add2(e, both(1.f));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(e.x));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(e.y));
  return e;
}

template <int LPR>
__device__ __forceinline__ float lanes_sum(float x) {
#pragma unroll
  for (int off = LPR / 2; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

template <int N>
__device__ __forceinline__ void zero_pairs(float2 (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = both(0.f);
}

constexpr int kGnThreads = 256;

// Where a thread's row stands, and whether it is to be read.  Index: 32 bits where every offset
// of the call fits, which takes a fifth of the kernels' instructions away.
template <typename Index>
struct GatedAt {
  Index row, gate;  // gate: offset of the row's gate
  bool in, valid;
  __device__ __forceinline__ GatedAt(const GatedNormParams& p, Index r, int d) : row(r), gate(r * d) {
    in = valid = r < (Index)p.rows;
    if (in && p.by_token) {  // the gate is strided, or rows may be padding
      const Index tok = p.H.div(r);
      valid = token_valid(tok, p.T, p.lengths);
      gate = tok * (Index)p.gate_stride + (r - tok * p.H.d) * d;
    }
  }
};

// the weight's eight elements of a lane
template <bool WIDE>
__device__ __forceinline__ void load_weight(const float* p, int lane, int lanes, float2 (&w)[4]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p + share<WIDE>(0, lane, lanes)));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p + share<WIDE>(4, lane, lanes)));
  w[0] = make_float2(a.x, a.y);
  w[1] = make_float2(a.z, a.w);
  w[2] = make_float2(b.x, b.y);
  w[3] = make_float2(b.z, b.w);
}

// LPR = d / 8 lanes per row, eight elements per lane; ROWS rows in flight per thread.
template <typename T, typename Index, int LPR, int GATE, int ROWS>
__global__ void __launch_bounds__(kGnThreads) gated_norm_fwd_kernel(GatedNormParams p) {
  constexpr int d = 8 * LPR, kPer = kGnThreads / LPR;
  constexpr bool kWide = sizeof(T) == 4;
  const int lane = threadIdx.x % LPR;
  struct {
    Raw8<T> o, g;
    Index row;
    bool in, valid;
  } r[ROWS];
#pragma unroll
  for (int u = 0; u < ROWS; ++u) {
    const GatedAt<Index> at(p, ((Index)blockIdx.x * ROWS + u) * kPer + threadIdx.x / LPR, d);
    r[u].row = at.row;
    r[u].in = at.in;
    r[u].valid = at.valid;
    if (at.valid) {
      r[u].o.template load<kWide>(static_cast<const T*>(p.o) + at.row * d, lane, LPR);
      if (GATE != kGateNone) r[u].g.template load<kWide>(static_cast<const T*>(p.gate) + at.gate, lane, LPR);
    } else {
      r[u].o.zero();
      r[u].g.zero();
    }
  }
  float2 w[4];
  load_weight<kWide>(p.weight, lane, LPR, w);
#pragma unroll
  for (int u = 0; u < ROWS; ++u) {
    float2 s = both(0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) s = fma2(r[u].o.get(i), r[u].o.get(i), s);
    const float rstd = rsqrtf(lanes_sum<LPR>(s.x + s.y) * (1.f / d) + p.eps);
    if (!r[u].in) continue;
    float2 y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[i] = mul2(mul2(r[u].o.get(i), both(rstd)), w[i]);
      if (GATE != kGateNone) {
        const float2 g = r[u].g.get(i), sg = sigmoid2<T>(g);
        y[i] = mul2(y[i], GATE == kGateSilu ? mul2(g, sg) : sg);
      }
    }
    // a weight need not be finite (asked of the call first: without that fp32 rows of 128 take 49 us, not 47)
    if (p.lengths && !r[u].valid) zero_pairs(y);
    store_shared8<kWide>(static_cast<T*>(p.y) + r[u].row * d, lane, LPR, d, y);
  }
}

// Persistent blocks: a thread keeps its eight columns for all its rows, so the weight's
// gradient is summed in registers, then over the block in shared memory.  The next two rows
// are on their way while one is worked on.
constexpr int kStages = 3;

template <typename T, typename Index, int LPR, int GATE>
__global__ void __launch_bounds__(kGnThreads, 4) gated_norm_bwd_kernel(GatedNormParams p) {
  constexpr int d = 8 * LPR, kPer = kGnThreads / LPR, kPieces = Raw8<T>::kPieces;
  constexpr bool kWide = sizeof(T) == 4;
  extern __shared__ __align__(16) char ring_smem[];
  Ring<3 * kPieces, kStages> ring(ring_smem);
  const int lane = threadIdx.x % LPR;
  const Index rows = (Index)p.rows, stride = (Index)gridDim.x * kPer;
  Index row = (Index)blockIdx.x * kPer + threadIdx.x / LPR;
  uint32_t flags = 0;  // bit k: the row k sets ahead is to be read
  auto fetch = [&](int ahead) {
    const GatedAt<Index> at(p, row + ahead * stride, d);
    const T *o = static_cast<const T*>(p.o), *dy = static_cast<const T*>(p.dy), *g = static_cast<const T*>(p.gate);
    const int n = at.valid ? d : 0;
    flags |= (uint32_t)at.valid << ahead;
    ring.template copy<kWide>(ahead, 0, o + at.row * d, lane, LPR, n, o);
    ring.template copy<kWide>(ahead, kPieces, dy + at.row * d, lane, LPR, n, o);
    if (GATE != kGateNone) ring.template copy<kWide>(ahead, 2 * kPieces, g + at.gate, lane, LPR, n, o);
    ring.commit();
  };
  launch_dependents();
#pragma unroll
  for (int ahead = 0; ahead < kStages - 1; ++ahead) fetch(ahead);
  float2 w[4], dw[4];
  load_weight<kWide>(p.weight, lane, LPR, w);
#pragma unroll
  for (int i = 0; i < 4; ++i) dw[i] = both(0.f);
  // the trip count is the same for the whole block
  for (Index base = (Index)blockIdx.x * kPer; base < rows; base += stride, row += stride, flags >>= 1) {
    ring.wait();
    const bool valid = flags & 1;
    T *d_o_row = static_cast<T*>(p.y) + row * d, *dg_row = static_cast<T*>(p.d_gate) + row * d;
    if (!__any_sync(0xffffffffu, valid)) {  // a warp of padding
      fetch(kStages - 1);
      ring.advance();
      const float2 zero[4] = {both(0.f), both(0.f), both(0.f), both(0.f)};
      if (row < rows) store_shared8<kWide>(d_o_row, lane, LPR, d, zero);
      if (GATE != kGateNone && row < rows) store_shared8<kWide>(dg_row, lane, LPR, d, zero);
      continue;
    }
    struct {
      Raw8<T> o, dy, g;
    } cur;
    cur.o = ring.template read<T>(0);
    cur.dy = ring.template read<T>(kPieces);
    if (GATE != kGateNone) cur.g = ring.template read<T>(2 * kPieces);
    fetch(kStages - 1);  // into the set that the previous row has been through
    ring.advance();
    float2 s = both(0.f), c = both(0.f), dg[4], t[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 o = cur.o.get(i), dy = cur.dy.get(i);
      s = fma2(o, o, s);
      t[i] = dy;
      if (GATE != kGateNone) {
        const float2 g = cur.g.get(i), sg = sigmoid2<T>(g);
        const float2 rest = fma2(sg, both(-1.f), both(1.f));  // 1 - sg
        if (GATE == kGateSilu) {
          dg[i] = mul2(dy, mul2(sg, fma2(g, rest, both(1.f))));  // times xh w below
          t[i] = mul2(dy, mul2(g, sg));
        } else {
          dg[i] = mul2(dy, mul2(sg, rest));
          t[i] = mul2(dy, sg);
        }
      }
      c = fma2(mul2(t[i], w[i]), o, c);
    }
    const float r = rsqrtf(lanes_sum<LPR>(s.x + s.y) * (1.f / d) + p.eps);
    const float mean = lanes_sum<LPR>(c.x + c.y) * r * (1.f / d);
    if (row >= rows) continue;
    float2 d_o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 xh = mul2(cur.o.get(i), both(r));
      dw[i] = fma2(t[i], xh, dw[i]);
      d_o[i] = mul2(fma2(xh, both(-mean), mul2(t[i], w[i])), both(r));
      if (GATE != kGateNone) dg[i] = mul2(dg[i], mul2(xh, w[i]));
    }
    // padding was read as zero and adds nothing to dw; a weight need not be finite
    if (!valid) {
      zero_pairs(d_o);
      if (GATE != kGateNone) zero_pairs(dg);
    }
    store_shared8<kWide>(d_o_row, lane, LPR, d, d_o);
    if (GATE != kGateNone) store_shared8<kWide>(dg_row, lane, LPR, d, dg);
  }
  ring.drain();
  __shared__ float sum[kPer][d];
#pragma unroll
  for (int e = 0; e < 8; ++e) sum[threadIdx.x / LPR][share<kWide>(e, lane, LPR)] = e & 1 ? dw[e / 2].y : dw[e / 2].x;
  __syncthreads();
  for (int c = threadIdx.x; c < d; c += kGnThreads) {
    float s = 0.f;
    for (int i = 0; i < kPer; ++i) s += sum[i][c];
    (gridDim.x == 1 ? p.d_weight : p.part + (size_t)blockIdx.x * d)[c] = s;
  }
}

// ------------------------------------------------------------------------------ block norm
// A group of tpr threads holds a row, E columns per thread: tpr is a power of two up to 32,
// or a multiple of 32.  MAP: kEven8 in 16-bit rows where D is a multiple of 8, kEven4 with an
// fp32 stream where it is one of 4 (the threads share 8 tpr columns at a time); kOdd otherwise:
// one column per access, consecutive threads on consecutive columns.
enum Map { kOdd = 0, kEven8 = 1, kEven4 = 2 };

template <int MAP>
__device__ __forceinline__ int column(int e, int gt, int tpr) {
  return MAP == kOdd ? gt + e * tpr : e / 8 * 8 * tpr + share<MAP == kEven4>(e % 8, gt, tpr);
}

// Eight of a thread's columns, as pairs.
struct Piece {
  float2 v[4];
};

// A thread's E columns of one row, one column per access; what is not `ok` or behind column D
// reads as zero.
template <typename T, int E>
struct Row {
  float w[E];
  __device__ __forceinline__ void load(const T* p, int gt, int tpr, int D, bool ok) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = column<kOdd>(e, gt, tpr);
      w[e] = ok && c < D ? load1(p + c) : 0.f;
    }
  }
  __device__ __forceinline__ Piece piece(int j) const {
    Piece r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.v[i] = make_float2(w[8 * j + 2 * i], w[8 * j + 2 * i + 1]);
    return r;
  }
};

// The same in pieces of eight through the thread's ring: a row's copies into the set `ahead`
// sets behind the next one to be read, from its slot `at` on, and a piece of the current set.
constexpr int kBnStages = 2;  // the next row is on its way while one is worked on

template <int MAP, typename T, int E, int N>
__device__ __forceinline__ void copy_row(Ring<N, kBnStages>& ring, int ahead, int at, const void* from, long long row,
                                         const BlockNormParams& p, int gt, bool ok) {
  const T* src = static_cast<const T*>(from) + row * p.D;
#pragma unroll
  for (int j = 0; j < E / 8; ++j) {
    const int c = 8 * j * p.tpr;
    ring.template copy<MAP == kEven4>(ahead, at + j * Raw8<T>::kPieces, src + c, gt, p.tpr, ok ? p.D - c : 0, p.x);
  }
}
template <typename T, int N>
__device__ __forceinline__ Piece ring_piece(const Ring<N, kBnStages>& ring, int at, int j) {
  const Raw8<T> r = ring.template read<T>(at + j * Raw8<T>::kPieces);
  return {{r.get(0), r.get(1), r.get(2), r.get(3)}};
}

template <int E, int MAP, typename T>
__device__ __forceinline__ void store_row(T* p, int gt, int tpr, int D, const float2 (&x)[E / 2]) {
  if constexpr (MAP == kOdd) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = column<kOdd>(e, gt, tpr);
      if (c < D) st1<T>(p + c, e & 1 ? x[e / 2].y : x[e / 2].x);
    }
  } else {
#pragma unroll
    for (int j = 0; j < E / 8; ++j) {
      const float2 v[4] = {x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]};
      store_shared8<MAP == kEven4>(p + 8 * j * tpr, gt, tpr, D - 8 * j * tpr, v);
    }
  }
}

// Padding.  A row of it was read as zeros, but the operations on zeros do not give zeros under a vector
// that is not finite, nor leave the vectors' gradients alone.  With the ring and rows of whole warps
// (columns per thread above 8, see BlockShape) a group goes from one row that is no padding to the
// next, and sets its rows of padding to zero in the end.  Rows that share a warp go together, and
// without the ring a branch before the row's use would part it from its loads (2991 x 1001 in fp32,
// forward: 27 us instead of 15): there a row's results are replaced by zeros.
template <int E, int MAP>
__device__ constexpr bool pass_padding() { return E > 8 && MAP != kOdd; }

// Number of a row: 32 bits for rows of more than 256 columns, of which no device holds 2^31.
template <int E, int MAP>
using RowIndex = typename std::conditional<pass_padding<E, MAP>(), uint32_t, long long>::type;

// The first of the rows row, row + stride, ... that is no padding, or one behind the last.
template <typename R>
__device__ __forceinline__ R next_row(const BlockNormParams& p, R row, R stride) {
  if (p.lengths)
    while (row < (R)p.rows && !token_valid(row, p.T, p.lengths)) row += stride;
  return row;
}

// Zeros into the rows of padding of this thread's group.  Last, and from the kernel's parameters alone:
// the loop over the other rows has no register to spare for it.
template <int E, int MAP, typename X, typename A>
__device__ __forceinline__ void zero_padding(const BlockNormParams& p, bool x_out, bool h) {
  if (!p.lengths) return;
  using R = RowIndex<E, MAP>;
  const int gt = threadIdx.x % p.tpr;
  float2 x[E / 2];
  zero_pairs(x);
  for (R row = (R)blockIdx.x * p.groups + threadIdx.x / p.tpr; row < (R)p.rows; row += (R)gridDim.x * p.groups) {
    if (token_valid(row, p.T, p.lengths)) continue;
    if (x_out) store_row<E, MAP>(static_cast<X*>(p.x_out) + (long long)row * p.D, gt, p.tpr, p.D, x);
    if (h) store_row<E, MAP>(static_cast<A*>(p.h) + (long long)row * p.D, gt, p.tpr, p.D, x);
  }
}

// Per-channel vectors live in shared memory, in the order in which a group's threads read
// them: a warp's 16-byte reads of four columns are consecutive.
template <int MAP>
__device__ __forceinline__ int vec_slot(int c, int tpr) {
  if (MAP != kEven8) return c;
  const int j = c / (8 * tpr), r = c - j * 8 * tpr;  // r = 8 gt + 4 half + i
  return ((2 * j + (r >> 2 & 1)) * tpr + (r >> 3)) * 4 + (r & 3);
}
// n = tpr * E slots of p (or `other`) times `factor`; zero behind column D
template <int MAP>
__device__ __forceinline__ void stage_vec(float* sv, const float* p, int D, int n, int tpr, float other, float factor) {
  for (int c = threadIdx.x; c < n; c += blockDim.x)
    sv[vec_slot<MAP>(c, tpr)] = c < D ? (p ? __ldg(p + c) : other) * factor : 0.f;
}
// piece j of a staged vector
template <int MAP>
__device__ __forceinline__ Piece vec_piece(const float* sv, int j, int gt, int tpr) {
  Piece r;
  sv += 8 * j * tpr;
  if (MAP == kOdd) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      r.v[i] = make_float2(sv[column<kOdd>(2 * i, gt, tpr)], sv[column<kOdd>(2 * i + 1, gt, tpr)]);
  } else {  // both orders: four columns of every thread, then the next four
    const float4 a = *reinterpret_cast<const float4*>(sv + 4 * gt), b = *reinterpret_cast<const float4*>(sv + 4 * (tpr + gt));
    r.v[0] = make_float2(a.x, a.y);
    r.v[1] = make_float2(a.z, a.w);
    r.v[2] = make_float2(b.x, b.y);
    r.v[3] = make_float2(b.z, b.w);
  }
  return r;
}

// Sum of each of the N values over the group, for every thread of it.  Groups of more than
// one warp (at most kBnGroups of them in a block) meet at a named barrier of their own; `buf`
// alternates between two shared arrays, so that one barrier per reduction is enough.
constexpr int kBnThreads = 512;  // most threads of a group
constexpr int kBnGroups = 4;     // most groups of more than one warp in a block

__device__ __forceinline__ void group_barrier(int group, int threads) {
  // constant barrier numbers: a variable one would reserve all sixteen
  if (group == 0) asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");
  else if (group == 1) asm volatile("bar.sync 2, %0;" ::"r"(threads) : "memory");
  else if (group == 2) asm volatile("bar.sync 3, %0;" ::"r"(threads) : "memory");
  else asm volatile("bar.sync 4, %0;" ::"r"(threads) : "memory");
}

// Sums of four values over a warp, value k in the lanes of 8 k .. 8 k + 7: halves of the lanes
// exchange values first, which takes 6 shuffles instead of 20.
__device__ __forceinline__ float warp_sum4(float a, float b, float c, float d) {
  const int lane = threadIdx.x % 32;
  const bool hi = lane & 16, odd = lane & 8;
  const float u = (hi ? c : a) + __shfl_xor_sync(0xffffffffu, hi ? a : c, 16);
  const float v = (hi ? d : b) + __shfl_xor_sync(0xffffffffu, hi ? b : d, 16);
  float x = (odd ? v : u) + __shfl_xor_sync(0xffffffffu, odd ? u : v, 8);
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

struct GroupSum {
  float4 (*buf)[2][kBnThreads / 32];  // [group][parity][warp]
  int parity = 0;
  template <int N>  // 1 to 4
  __device__ __forceinline__ void run(float (&x)[N], int group, int gt, int tpr) {
    if (tpr <= 32) {
      for (int off = tpr / 2; off > 0; off >>= 1) {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] += __shfl_xor_sync(0xffffffffu, x[i], off);
      }
      return;
    }
    float* mine = reinterpret_cast<float*>(&buf[group][parity][gt / 32]);
    if (N == 1) {
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) x[0] += __shfl_xor_sync(0xffffffffu, x[0], off);
      if (gt % 32 == 0) mine[0] = x[0];
    } else {
      const float s = warp_sum4(x[0], x[1 % N], N > 2 ? x[2 % N] : 0.f, N > 3 ? x[3 % N] : 0.f);
      if (gt % 8 == 0) mine[gt % 32 / 8] = s;
    }
    group_barrier(group, tpr);
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int w = 0; w < tpr / 32; ++w) {
      const float4 v = buf[group][parity][w];
      t.x += v.x;
      if (N > 1) t.y += v.y;
      if (N > 2) t.z += v.z;
      if (N > 3) t.w += v.w;
    }
    x[0] = t.x;
    if (N > 1) x[1 % N] = t.y;
    if (N > 2) x[2 % N] = t.z;
    if (N > 3) x[3 % N] = t.w;
    parity ^= 1;
  }
};

// The rows of a group of the backward, piece by piece; padding reads as zero.  Vectorised
// form: through the thread's ring.
template <typename X, typename A, int E, int MAP, bool Y>
struct BwdRows {
  static constexpr int kX = Raw8<X>::kPieces * E / 8, kA = Raw8<A>::kPieces * E / 8, kAll = 2 * kX + (Y ? 2 : 1) * kA;
  const BlockNormParams& p;
  int gt;
  Ring<kAll, kBnStages> ring;
  bool valid, next_valid;  // whether the row at hand, and the one behind it, exist and are no padding
  __device__ __forceinline__ BwdRows(const BlockNormParams& p_, int gt_, void* smem) : p(p_), gt(gt_), ring(smem) {}
  __device__ __forceinline__ void fetch(int ahead, long long row) {
    const bool ok = next_valid = row < p.rows && (pass_padding<E, MAP>() || token_valid(row, p.T, p.lengths));
    copy_row<MAP, X, E>(ring, ahead, 0, p.x, row, p, gt, ok);
    copy_row<MAP, X, E>(ring, ahead, kX, p.dx_in ? p.dx_in : p.x, row, p, gt, ok && p.dx_in);
    copy_row<MAP, A, E>(ring, ahead, 2 * kX, p.dh, row, p, gt, ok);
    if (Y) copy_row<MAP, A, E>(ring, ahead, 2 * kX + kA, p.y, row, p, gt, ok);
    ring.commit();
  }
  __device__ __forceinline__ void start(long long row) { fetch(0, row); }
  // the row's set is complete; the one behind it, which the previous row has been through, is filled
  __device__ __forceinline__ void take(long long, long long next) {
    ring.wait();
    valid = next_valid;
    fetch(1, next);
  }
  __device__ __forceinline__ void leave() { ring.advance(); }
  __device__ __forceinline__ void finish() { ring.drain(); }
  __device__ __forceinline__ Piece x(int j) const { return ring_piece<X>(ring, 0, j); }
  __device__ __forceinline__ Piece dx(int j) const { return ring_piece<X>(ring, kX, j); }
  __device__ __forceinline__ Piece dh(int j) const { return ring_piece<A>(ring, 2 * kX, j); }
  __device__ __forceinline__ Piece y(int j) const { return ring_piece<A>(ring, 2 * kX + kA, j); }
};

// Other widths: one column per access, straight into registers.
template <typename X, typename A, int E, bool Y>
struct BwdRows<X, A, E, kOdd, Y> {
  static constexpr int kAll = 0;
  const BlockNormParams& p;
  int gt;
  Row<X, E> rx, rdx;
  Row<A, E> rdh, ry;
  bool valid;
  __device__ __forceinline__ BwdRows(const BlockNormParams& p_, int gt_, void*) : p(p_), gt(gt_) {}
  __device__ __forceinline__ void start(long long) {}
  __device__ __forceinline__ void take(long long row, long long) {
    const bool ok = valid = row < p.rows && token_valid(row, p.T, p.lengths);
    rx.load(static_cast<const X*>(p.x) + row * p.D, gt, p.tpr, p.D, ok);
    rdh.load(static_cast<const A*>(p.dh) + row * p.D, gt, p.tpr, p.D, ok);
    rdx.load(static_cast<const X*>(p.dx_in) + row * p.D, gt, p.tpr, p.D, ok && p.dx_in);
    if (Y) ry.load(static_cast<const A*>(p.y) + row * p.D, gt, p.tpr, p.D, ok);
  }
  __device__ __forceinline__ void leave() {}
  __device__ __forceinline__ void finish() {}
  __device__ __forceinline__ Piece x(int j) const { return rx.piece(j); }
  __device__ __forceinline__ Piece dx(int j) const { return rdx.piece(j); }
  __device__ __forceinline__ Piece dh(int j) const { return rdh.piece(j); }
  __device__ __forceinline__ Piece y(int j) const { return ry.piece(j); }
};

// The rows of a group of the forward: as BwdRows, with x and y.
template <typename X, typename A, int E, int MAP, bool DELTA>
struct FwdRows {
  static constexpr int kX = Raw8<X>::kPieces * E / 8, kA = Raw8<A>::kPieces * E / 8, kAll = kX + (DELTA ? kA : 0);
  const BlockNormParams& p;
  int gt;
  Ring<kAll, kBnStages> ring;
  bool valid, next_valid;
  __device__ __forceinline__ FwdRows(const BlockNormParams& p_, int gt_, void* smem) : p(p_), gt(gt_), ring(smem) {}
  __device__ __forceinline__ void fetch(int ahead, long long row) {
    const bool ok = next_valid = row < p.rows && (pass_padding<E, MAP>() || token_valid(row, p.T, p.lengths));
    copy_row<MAP, X, E>(ring, ahead, 0, p.x, row, p, gt, ok);
    if (DELTA) copy_row<MAP, A, E>(ring, ahead, kX, p.y, row, p, gt, ok);
    ring.commit();
  }
  __device__ __forceinline__ void start(long long row) { fetch(0, row); }
  __device__ __forceinline__ void take(long long, long long next) {
    ring.wait();
    valid = next_valid;
    fetch(1, next);
  }
  __device__ __forceinline__ void leave() { ring.advance(); }
  __device__ __forceinline__ void finish() { ring.drain(); }
  __device__ __forceinline__ Piece x(int j) const { return ring_piece<X>(ring, 0, j); }
  __device__ __forceinline__ Piece y(int j) const { return ring_piece<A>(ring, kX, j); }
};

template <typename X, typename A, int E, bool DELTA>
struct FwdRows<X, A, E, kOdd, DELTA> {
  static constexpr int kAll = 0;
  const BlockNormParams& p;
  int gt;
  Row<X, E> rx;
  Row<A, E> ry;
  bool valid;
  __device__ __forceinline__ FwdRows(const BlockNormParams& p_, int gt_, void*) : p(p_), gt(gt_) {}
  __device__ __forceinline__ void start(long long) {}
  __device__ __forceinline__ void take(long long row, long long) {
    const bool ok = valid = row < p.rows && token_valid(row, p.T, p.lengths);
    rx.load(static_cast<const X*>(p.x) + row * p.D, gt, p.tpr, p.D, ok);
    if (DELTA) ry.load(static_cast<const A*>(p.y) + row * p.D, gt, p.tpr, p.D, ok);
  }
  __device__ __forceinline__ void leave() {}
  __device__ __forceinline__ void finish() {}
  __device__ __forceinline__ Piece x(int j) const { return rx.piece(j); }
  __device__ __forceinline__ Piece y(int j) const { return ry.piece(j); }
};

// Most threads of a block and blocks of an SM, by columns per thread (registers: about 2 E for
// the row at hand, and 3 E for the backward's column sums).
__host__ __device__ constexpr int fwd_threads(int E) { return E == 16 ? 512 : 256; }
__host__ __device__ constexpr int fwd_blocks(int E) { return E == 8 ? 5 : E == 16 ? 2 : E == 24 ? 3 : 2; }

template <typename X, typename A, int E, int MAP, bool DELTA, bool POST>
__global__ void __launch_bounds__(fwd_threads(E), fwd_blocks(E)) block_norm_fwd_kernel(BlockNormParams p) {
  constexpr int P = E / 2;
  __shared__ float4 buf[kBnGroups][2][kBnThreads / 32];
  extern __shared__ __align__(16) float vecs[];  // weight, k, post_weight: tpr * E each; behind them the ring
  const int tpr = p.tpr, gt = threadIdx.x % tpr, group = threadIdx.x / tpr, D = p.D, n = tpr * E;
  GroupSum sum{buf};
  FwdRows<X, A, E, MAP, DELTA> rows(p, gt, vecs + (1 + DELTA + POST) * n);
  constexpr bool kPass = pass_padding<E, MAP>();
  using R = RowIndex<E, MAP>;
  const R stride = (R)gridDim.x * p.groups, end = (R)p.rows;
  R row = (R)blockIdx.x * p.groups + group, next;
  if (kPass) row = next_row(p, row, stride);
  rows.start(row);
  stage_vec<MAP>(vecs, p.weight, D, n, tpr, 1.f, 1.f);
  if (DELTA) stage_vec<MAP>(vecs + n, p.scale, D, n, tpr, 1.f, p.res_scale);
  if (POST) stage_vec<MAP>(vecs + 2 * n, p.post_weight, D, n, tpr, 1.f, 1.f);
  __syncthreads();
  // rows that share a warp: the trip count is the same for the whole block
  for (R base = row - group; (kPass ? row : base) < end; base += stride, row = next) {
    next = kPass ? next_row<R>(p, row + stride, stride) : row + stride;
    rows.take(row, next);
    const bool in = kPass || row < end, valid = kPass || rows.valid;
    float2 x[P], q = both(0.f);
    float s[1], ry = 1.f;
    if (POST) {
#pragma unroll
      for (int j = 0; j < E / 8; ++j) {
        const Piece y = rows.y(j);
#pragma unroll
        for (int i = 0; i < 4; ++i) q = fma2(y.v[i], y.v[i], q);
      }
      s[0] = q.x + q.y;
      sum.run(s, group, gt, tpr);
      ry = rsqrtf(s[0] * p.inv_D + p.eps);
      q = both(0.f);
    }
#pragma unroll
    for (int j = 0; j < E / 8; ++j) {
      const Piece xj = rows.x(j);
      Piece y, k, wp;
      if (DELTA) {
        y = rows.y(j);
        k = vec_piece<MAP>(vecs + n, j, gt, tpr);
      }
      if (POST) wp = vec_piece<MAP>(vecs + 2 * n, j, gt, tpr);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float2& v = x[4 * j + i];
        v = xj.v[i];
        if (DELTA) v = fma2(POST ? mul2(mul2(y.v[i], both(ry)), wp.v[i]) : y.v[i], k.v[i], v);
        q = fma2(v, v, q);
      }
    }
    if (!valid) zero_pairs(x);
    if (DELTA && in) store_row<E, MAP>(static_cast<X*>(p.x_out) + (long long)row * D, gt, tpr, D, x);
    s[0] = q.x + q.y;
    sum.run(s, group, gt, tpr);
    const float r = rsqrtf(s[0] * p.inv_D + p.eps);
#pragma unroll
    for (int j = 0; j < E / 8; ++j) {
      const Piece w = vec_piece<MAP>(vecs, j, gt, tpr);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[4 * j + i] = mul2(mul2(x[4 * j + i], both(r)), w.v[i]);
    }
    if (!valid) zero_pairs(x);
    if (in) store_row<E, MAP>(static_cast<A*>(p.h) + (long long)row * D, gt, tpr, D, x);
    rows.leave();
  }
  rows.finish();
  if (kPass) zero_padding<E, MAP, X, A>(p, DELTA, true);
}

// Most threads of a block of the backward.  One block fills an SM: fewer blocks leave fewer
// partial column sums.
__host__ __device__ constexpr int bwd_threads(int E, bool vec) {
  return vec ? (E == 8 ? 640 : E == 16 ? 512 : E == 24 ? 384 : 256) : 512;
}

// Persistent blocks: a thread keeps its columns for all its rows, so the vectors' gradients
// are summed in registers.  SCALE: there is a per-channel scale whose gradient is wanted.
template <typename X, typename A, int E, int MAP, bool DELTA, bool POST, bool SCALE>
__global__ void __launch_bounds__(bwd_threads(E, MAP != kOdd), 1)
    block_norm_bwd_kernel(BlockNormParams p) {
  constexpr int P = E / 2;
  constexpr bool Y = POST || SCALE;  // whether y is needed
  constexpr int N = POST ? 3 : 2;
  __shared__ float4 buf[kBnGroups][2][kBnThreads / 32];
  // weight, k, post_weight: tpr * E each; in the end the groups' column sums; behind them the ring
  extern __shared__ __align__(16) float vecs[];
  const int tpr = p.tpr, gt = threadIdx.x % tpr, group = threadIdx.x / tpr, D = p.D, n = tpr * E;
  GroupSum sum{buf};
  BwdRows<X, A, E, MAP, Y> rows(p, gt, vecs + max(3, p.groups) * n);
  launch_dependents();
  constexpr bool kPass = pass_padding<E, MAP>();
  using R = RowIndex<E, MAP>;
  const R stride = (R)gridDim.x * p.groups, end = (R)p.rows;
  R row = (R)blockIdx.x * p.groups + group, next;
  if (kPass) row = next_row(p, row, stride);
  rows.start(row);
  stage_vec<MAP>(vecs, p.weight, D, n, tpr, 1.f, 1.f);
  if (DELTA) stage_vec<MAP>(vecs + n, p.scale, D, n, tpr, 1.f, p.res_scale);
  if (POST) stage_vec<MAP>(vecs + 2 * n, p.post_weight, D, n, tpr, 1.f, 1.f);
  __syncthreads();
  float2 aw[P], ap[P], as[P];
#pragma unroll
  for (int i = 0; i < P; ++i) aw[i] = ap[i] = as[i] = both(0.f);
  // rows that share a warp: the trip count is the same for the whole block
  for (; (kPass ? row : row - group) < end; row = next) {
    next = kPass ? next_row<R>(p, row + stride, stride) : row + stride;
    rows.take(row, next);
    const bool in = kPass || row < end, valid = kPass || rows.valid;
    float s[N];
    float2 q0 = both(0.f), q1 = both(0.f), q2 = both(0.f);
#pragma unroll
    for (int j = 0; j < E / 8; ++j) {
      const Piece x = rows.x(j), dh = rows.dh(j), w = vec_piece<MAP>(vecs, j, gt, tpr);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        q0 = fma2(x.v[i], x.v[i], q0);
        q1 = fma2(mul2(dh.v[i], w.v[i]), x.v[i], q1);
      }
      if (POST) {
        const Piece y = rows.y(j);
#pragma unroll
        for (int i = 0; i < 4; ++i) q2 = fma2(y.v[i], y.v[i], q2);
      }
    }
    s[0] = q0.x + q0.y;
    s[1] = q1.x + q1.y;
    if (POST) s[N - 1] = q2.x + q2.y;
    sum.run(s, group, gt, tpr);
    const float r = rsqrtf(s[0] * p.inv_D + p.eps), mean = s[1] * r * p.inv_D;
    const float ry = POST ? rsqrtf(s[N - 1] * p.inv_D + p.eps) : 1.f;
    float2 dx[P], c2 = both(0.f);
#pragma unroll
    for (int j = 0; j < E / 8; ++j) {
      const Piece x = rows.x(j), dh = rows.dh(j), d = rows.dx(j), w = vec_piece<MAP>(vecs, j, gt, tpr);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 xh = mul2(x.v[i], both(r));
        aw[4 * j + i] = fma2(dh.v[i], xh, aw[4 * j + i]);
        dx[4 * j + i] = fma2(fma2(xh, both(-mean), mul2(dh.v[i], w.v[i])), both(r), d.v[i]);
      }
    }
    if (!valid) zero_pairs(dx);
    if (in) store_row<E, MAP>(static_cast<X*>(p.x_out) + (long long)row * D, gt, tpr, D, dx);
    if (DELTA) {
      if (valid) {
#pragma unroll
        for (int j = 0; j < E / 8; ++j) {
          const Piece k = vec_piece<MAP>(vecs + n, j, gt, tpr);
          Piece y, wp;
          if (Y) y = rows.y(j);
          if (POST) wp = vec_piece<MAP>(vecs + 2 * n, j, gt, tpr);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float2& d = dx[4 * j + i];
            if (POST) {
              const float2 yh = mul2(y.v[i], both(ry)), dz = mul2(d, k.v[i]);
              if (SCALE) as[4 * j + i] = fma2(d, mul2(yh, wp.v[i]), as[4 * j + i]);  // times res_scale at the end
              ap[4 * j + i] = fma2(dz, yh, ap[4 * j + i]);
              d = mul2(dz, wp.v[i]);
              c2 = fma2(d, yh, c2);
            } else {
              if (SCALE) as[4 * j + i] = fma2(d, y.v[i], as[4 * j + i]);
              d = mul2(d, k.v[i]);
            }
          }
        }
      }
      if (POST) {
        float c[1] = {c2.x + c2.y};
        sum.run(c, group, gt, tpr);
        const float my = -c[0] * p.inv_D * ry;
#pragma unroll
        for (int j = 0; j < E / 8; ++j) {
          const Piece y = rows.y(j);
#pragma unroll
          for (int i = 0; i < 4; ++i) dx[4 * j + i] = mul2(fma2(y.v[i], both(my), dx[4 * j + i]), both(ry));
        }
      }
      if (in) store_row<E, MAP>(static_cast<A*>(p.h) + (long long)row * D, gt, tpr, D, dx);
    }
    rows.leave();
  }
  rows.finish();
  // column sums of the block: one vector after the other through shared memory
  constexpr int kVec = 1 + (POST ? 1 : 0) + (SCALE ? 1 : 0);
#pragma unroll
  for (int v = 0; v < kVec; ++v) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float2 a = v == 0 ? aw[e / 2] : (POST && v == 1 ? ap[e / 2] : mul2(as[e / 2], both(p.res_scale)));
      vecs[group * n + column<MAP>(e, gt, tpr)] = e & 1 ? a.y : a.x;
    }
    __syncthreads();
    float* out = gridDim.x == 1 ? p.sums[v] : p.part + ((size_t)blockIdx.x * kVec + v) * D;
    for (int c = threadIdx.x; c < D; c += blockDim.x) {
      float t = 0.f;
      for (int g = 0; g < p.groups; ++g) t += vecs[g * n + c];
      out[c] = t;
    }
  }
  if (kPass) zero_padding<E, MAP, X, A>(p, true, DELTA);
}

// Eight columns (one 32-byte sector of a row) and 64 slices of the rows per block.
constexpr int kSumCols = 8, kSumSlices = 64;

__global__ void __launch_bounds__(kSumCols * kSumSlices) column_sum_kernel(ColumnSumParams p) {
  __shared__ float sm[kSumSlices][kSumCols];
  const int col = blockIdx.x * kSumCols + threadIdx.x % kSumCols, slice = threadIdx.x / kSumCols;
  const int n = p.nvec * p.D;
  float s = 0.f;
  wait_for_previous();
  if (col < n) {
#pragma unroll 8
    for (int b = slice; b < p.blocks; b += kSumSlices) s += p.part[(size_t)b * n + col];
  }
  sm[slice][threadIdx.x % kSumCols] = s;
  __syncthreads();
  if (slice == 0 && col < n) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < kSumSlices; ++i) t += sm[i][threadIdx.x];
    const int v = col / p.D;
    p.out[v][col - v * p.D] = t;
  }
}

// Dynamic shared memory of a block norm's block, beside 2 KB of static: the only one on its SM, or
// one of several that share the SM's 228 KB (each takes 1 KB more for itself).
constexpr size_t kMostSmem = 224 * 1024;
constexpr size_t smem_share(int blocks) { return 228 * 1024 / blocks - 3 * 1024; }

template <typename... Args>
cudaError_t launch_with_smem(void (*kernel)(Args...), size_t most, int blocks, int threads, size_t smem,
                             cudaStream_t stream, Args... args) {
  if (smem > 32 * 1024) {  // the kernel's limit is the same in every call: another thread may be launching it too
    const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    if (err != cudaSuccess) return err;
  }
  kernel<<<blocks, threads, smem, stream>>>(args...);
  return cudaGetLastError();
}

template <typename T, typename Index, int LPR>
cudaError_t gated_fwd_index(const GatedNormParams& p, int gate, cudaStream_t stream) {
  constexpr int kRows = sizeof(T) == 2 ? 4 : 2;
  const long long per = (long long)kRows * (kGnThreads / LPR);
  const int blocks = (int)((p.rows + per - 1) / per);
  if (gate == kGateNone)
    gated_norm_fwd_kernel<T, Index, LPR, kGateNone, kRows><<<blocks, kGnThreads, 0, stream>>>(p);
  else if (gate == kGateSilu)
    gated_norm_fwd_kernel<T, Index, LPR, kGateSilu, kRows><<<blocks, kGnThreads, 0, stream>>>(p);
  else
    gated_norm_fwd_kernel<T, Index, LPR, kGateSigmoid, kRows><<<blocks, kGnThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

// whether the offsets of a call, and of the rows that its last blocks would have, fit 32 bits
bool fits32(const GatedNormParams& p, int d) {
  const double toks = (double)p.rows / p.H.d + 65536;
  return toks * p.H.d * d < 2.0e9 && toks * p.gate_stride < 2.0e9 && p.rows < (1ll << 30);
}

template <typename T, int LPR>
cudaError_t gated_fwd_lanes(const GatedNormParams& p, int gate, cudaStream_t stream) {
  return fits32(p, 8 * LPR) ? gated_fwd_index<T, uint32_t, LPR>(p, gate, stream)
                            : gated_fwd_index<T, long long, LPR>(p, gate, stream);
}

template <typename T, typename Index, int LPR>
cudaError_t gated_bwd_index(const GatedNormParams& p, int gate, int blocks, cudaStream_t stream) {
  const size_t smem = Ring<3 * Raw8<T>::kPieces, kStages>::bytes(kGnThreads);
  if (gate == kGateNone)
    return launch_with_smem(gated_norm_bwd_kernel<T, Index, LPR, kGateNone>, smem, blocks, kGnThreads, smem, stream,
                            p);
  if (gate == kGateSilu)
    return launch_with_smem(gated_norm_bwd_kernel<T, Index, LPR, kGateSilu>, smem, blocks, kGnThreads, smem, stream,
                            p);
  return launch_with_smem(gated_norm_bwd_kernel<T, Index, LPR, kGateSigmoid>, smem, blocks, kGnThreads, smem, stream,
                          p);
}

template <typename T, int LPR>
cudaError_t gated_bwd_lanes(const GatedNormParams& p, int gate, int blocks, cudaStream_t stream) {
  return fits32(p, 8 * LPR) ? gated_bwd_index<T, uint32_t, LPR>(p, gate, blocks, stream)
                            : gated_bwd_index<T, long long, LPR>(p, gate, blocks, stream);
}

// How the block norm is cut: E columns per thread, tpr threads per row, `groups` rows at a time
// per block.  A warp holds a row of up to 1024 columns, so that no barrier stands between its
// sums (the 130M-LM backward with 96 threads a row and two barriers: 120 us; with a warp: 60).
// Widths that are not a multiple of 8 (4 with an fp32 stream), or whose rings would not fit the
// shared memory, take one column per access: 32509 x 769 in bf16 145 us forward and 232 backward, where
// 768 columns take 40 and 59; in fp32 100 and 176 against 76 and 116.
struct BlockShape {
  int E, tpr, groups;
  bool vec;
  BlockShape(int D, bool bwd, int x_bytes, int bytes) {
    const int arrays = (bwd ? 2 : 1) * (x_bytes + bytes);  // bytes of a column that the ring holds per row
    const size_t row = (size_t)((D + 1023) / 1024 * 1024) * (kBnStages * arrays);
    vec = D % (x_bytes == 4 ? 4 : 8) == 0 && row + (size_t)(D + 1023) / 1024 * 1024 * 12 <= kMostSmem;
    if (bwd) E = D <= 1024 && vec ? (D + 255) / 256 * 8 : vec ? 16 : D <= 4096 ? 8 : 16;
    else E = D <= 1024 ? (D + 255) / 256 * 8 : 16;
    const int t = (D + E - 1) / E, most = bwd ? bwd_threads(E, vec) : fwd_threads(E);
    tpr = E > 8 ? 32 : 1;  // pass_padding()
    while (tpr < 32 && tpr < t) tpr *= 2;
    if (t > 32) tpr = (t + 31) / 32 * 32;
    groups = most / tpr;
    if (tpr > 32 && groups > kBnGroups) groups = kBnGroups;
    if (vec) {  // a group's part of the rings and of the backward's column sums
      const size_t group = (size_t)tpr * E * (kBnStages * arrays + (bwd ? 4 : 0)), vecs = (size_t)tpr * E * 12;
      const size_t block = bwd ? kMostSmem : smem_share(fwd_blocks(E));
      if (vecs + groups * group > block) groups = block > vecs ? (int)((block - vecs) / group) : 1;
    }
    if (tpr < 32) groups -= groups % (32 / tpr);  // whole warps
    if (groups < 1) groups = 1;
  }
};

template <typename X, typename A, int E, int MAP, bool DELTA, bool POST>
cudaError_t block_fwd_kernel(const BlockNormParams& p, int blocks, cudaStream_t stream) {
  const int threads = p.tpr * p.groups;
  const size_t vecs = (size_t)(1 + DELTA + POST) * p.tpr * E * 4;
  const size_t ring = (size_t)FwdRows<X, A, E, MAP, DELTA>::kAll * 16 * kBnStages * threads;
  return launch_with_smem(block_norm_fwd_kernel<X, A, E, MAP, DELTA, POST>, kMostSmem, blocks, threads, vecs + ring,
                          stream, p);
}

template <typename X, typename A, int E, int MAP>
cudaError_t block_fwd_cols(const BlockNormParams& p, int blocks, cudaStream_t stream) {
  if (!p.y) return block_fwd_kernel<X, A, E, MAP, false, false>(p, blocks, stream);
  if (!p.post_weight) return block_fwd_kernel<X, A, E, MAP, true, false>(p, blocks, stream);
  return block_fwd_kernel<X, A, E, MAP, true, true>(p, blocks, stream);
}

template <typename X, typename A, int E, int MAP, bool DELTA, bool POST, bool SCALE>
cudaError_t block_bwd_kernel(const BlockNormParams& p, int blocks, cudaStream_t stream) {
  const int threads = p.tpr * p.groups;
  const size_t vecs = (size_t)(p.groups > 3 ? p.groups : 3) * p.tpr * E * 4;
  const size_t ring = (size_t)BwdRows<X, A, E, MAP, POST || SCALE>::kAll * 16 * kBnStages * threads;
  return launch_with_smem(block_norm_bwd_kernel<X, A, E, MAP, DELTA, POST, SCALE>, kMostSmem, blocks, threads,
                          vecs + ring, stream, p);
}

template <typename X, typename A, int E, int MAP>
cudaError_t block_bwd_cols(const BlockNormParams& p, int blocks, cudaStream_t stream) {
  if (!p.y) return block_bwd_kernel<X, A, E, MAP, false, false, false>(p, blocks, stream);
  if (!p.post_weight && !p.scale) return block_bwd_kernel<X, A, E, MAP, true, false, false>(p, blocks, stream);
  if (!p.post_weight) return block_bwd_kernel<X, A, E, MAP, true, false, true>(p, blocks, stream);
  if (!p.scale) return block_bwd_kernel<X, A, E, MAP, true, true, false>(p, blocks, stream);
  return block_bwd_kernel<X, A, E, MAP, true, true, true>(p, blocks, stream);
}

template <typename X, typename A>
cudaError_t block_norm_types(BlockNormParams p, bool bwd, cudaStream_t stream) {
  const BlockShape s(p.D, bwd, sizeof(X), sizeof(A));
  p.tpr = s.tpr;
  p.groups = s.groups;
  const int blocks = block_norm_blocks(p.rows, p.D, bwd, sizeof(X), sizeof(A));
  constexpr int kEven = sizeof(X) == 4 ? kEven4 : kEven8;
  if (bwd && !s.vec)
    return s.E == 8 ? block_bwd_cols<X, A, 8, kOdd>(p, blocks, stream) : block_bwd_cols<X, A, 16, kOdd>(p, blocks, stream);
  if (bwd) switch (s.E) {
      case 8: return block_bwd_cols<X, A, 8, kEven>(p, blocks, stream);
      case 16: return block_bwd_cols<X, A, 16, kEven>(p, blocks, stream);
      case 24: return block_bwd_cols<X, A, 24, kEven>(p, blocks, stream);
      default: return block_bwd_cols<X, A, 32, kEven>(p, blocks, stream);
    }
  if (!s.vec) switch (s.E) {
      case 8: return block_fwd_cols<X, A, 8, kOdd>(p, blocks, stream);
      case 16: return block_fwd_cols<X, A, 16, kOdd>(p, blocks, stream);
      case 24: return block_fwd_cols<X, A, 24, kOdd>(p, blocks, stream);
      default: return block_fwd_cols<X, A, 32, kOdd>(p, blocks, stream);
    }
  switch (s.E) {
    case 8: return block_fwd_cols<X, A, 8, kEven>(p, blocks, stream);
    case 16: return block_fwd_cols<X, A, 16, kEven>(p, blocks, stream);
    case 24: return block_fwd_cols<X, A, 24, kEven>(p, blocks, stream);
    default: return block_fwd_cols<X, A, 32, kEven>(p, blocks, stream);
  }
}

}  // namespace

int block_norm_blocks(long long rows, int D, bool bwd, int x_bytes, int bytes) {
  const BlockShape s(D, bwd, x_bytes, bytes);
  const int threads = s.tpr * s.groups, fit = bwd ? 1 : fwd_blocks(s.E) * fwd_threads(s.E) / threads;
  const long long need = (rows + s.groups - 1) / s.groups, most = (long long)kSMs * (fit < 1 ? 1 : fit);
  return (int)(need < most ? need : most);
}

cudaError_t launch_column_sum(const ColumnSumParams& p, cudaStream_t stream) {
  const int cols = p.nvec * p.D;
  return launch_chained(column_sum_kernel, dim3((cols + kSumCols - 1) / kSumCols), kSumCols * kSumSlices, 0, stream, p);
}

cudaError_t launch_gated_norm_fwd(const GatedNormParams& p, int d, int gate, int dtype, cudaStream_t stream) {
  if (dtype == PRISM_FP32) switch (d) {
      case 16: return gated_fwd_lanes<float, 2>(p, gate, stream);
      case 32: return gated_fwd_lanes<float, 4>(p, gate, stream);
      case 64: return gated_fwd_lanes<float, 8>(p, gate, stream);
      default: return gated_fwd_lanes<float, 16>(p, gate, stream);
    }
  switch (d) {
    case 16: return gated_fwd_lanes<__nv_bfloat16, 2>(p, gate, stream);
    case 32: return gated_fwd_lanes<__nv_bfloat16, 4>(p, gate, stream);
    case 64: return gated_fwd_lanes<__nv_bfloat16, 8>(p, gate, stream);
    default: return gated_fwd_lanes<__nv_bfloat16, 16>(p, gate, stream);
  }
}

cudaError_t launch_gated_norm_bwd(const GatedNormParams& p, int d, int gate, int dtype, cudaStream_t stream) {
  const int blocks = gated_norm_bwd_blocks(p.rows, d);
  cudaError_t err;
  if (dtype == PRISM_FP32) switch (d) {
      case 16: err = gated_bwd_lanes<float, 2>(p, gate, blocks, stream); break;
      case 32: err = gated_bwd_lanes<float, 4>(p, gate, blocks, stream); break;
      case 64: err = gated_bwd_lanes<float, 8>(p, gate, blocks, stream); break;
      default: err = gated_bwd_lanes<float, 16>(p, gate, blocks, stream);
    }
  else switch (d) {
      case 16: err = gated_bwd_lanes<__nv_bfloat16, 2>(p, gate, blocks, stream); break;
      case 32: err = gated_bwd_lanes<__nv_bfloat16, 4>(p, gate, blocks, stream); break;
      case 64: err = gated_bwd_lanes<__nv_bfloat16, 8>(p, gate, blocks, stream); break;
      default: err = gated_bwd_lanes<__nv_bfloat16, 16>(p, gate, blocks, stream);
    }
  if (err != cudaSuccess || blocks == 1) return err;
  ColumnSumParams c{p.part, {p.d_weight, nullptr, nullptr}, blocks, 1, d};
  return launch_column_sum(c, stream);
}

cudaError_t launch_block_norm(const BlockNormParams& p, bool bwd, int x_dtype, int dtype, cudaStream_t stream) {
  const int x_bytes = x_dtype == PRISM_FP32 ? 4 : 2, bytes = dtype == PRISM_FP32 ? 4 : 2;
  const cudaError_t err = x_bytes == 2   ? block_norm_types<__nv_bfloat16, __nv_bfloat16>(p, bwd, stream)
                          : bytes == 2 ? block_norm_types<float, __nv_bfloat16>(p, bwd, stream)
                                       : block_norm_types<float, float>(p, bwd, stream);
  const int blocks = block_norm_blocks(p.rows, p.D, bwd, x_bytes, bytes);
  if (err != cudaSuccess || !bwd || blocks == 1) return err;
  const int nvec = 1 + (p.post_weight ? 1 : 0) + (p.scale ? 1 : 0);
  ColumnSumParams c{p.part, {p.sums[0], p.sums[1], p.sums[2]}, blocks, nvec, p.D};
  return launch_column_sum(c, stream);
}

}  // namespace prism
