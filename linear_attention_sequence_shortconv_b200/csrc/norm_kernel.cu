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
#include "rowops.cuh"

namespace prism {

// Blocks of the persistent kernels; the backward ones set the number of partial column sums.
int gated_norm_bwd_blocks(long long rows, int d) {
  const long long per = 256 / (d / 8), need = (rows + per - 1) / per;
  return (int)(need < 4 * kSMs ? need : 4 * kSMs);
}
int block_norm_blocks(long long rows, int D, bool bwd);

namespace {

enum { kGateNone = 0, kGateSilu = 1, kGateSigmoid = 2 };

// 1 / (1 + e^-g).  fp32 outputs take the accurate exponential and division; for bf16 outputs
// the fast forms' error (a few units of 2^-23 of the exponent's argument) is far below the
// rounding to 8 bits.
template <typename T>
__device__ __forceinline__ float sigmoid(float g);
template <>
__device__ __forceinline__ float sigmoid<float>(float g) { return 1.f / (1.f + expf(-g)); }
template <>
__device__ __forceinline__ float sigmoid<__nv_bfloat16>(float g) { return __fdividef(1.f, 1.f + __expf(-g)); }

template <int LPR>
__device__ __forceinline__ float lanes_sum(float x) {
#pragma unroll
  for (int off = LPR / 2; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

constexpr int kGnThreads = 256;
constexpr int kGnRows = 2;  // rows in flight per thread

// LPR = d / 8 lanes per row, eight elements per lane.
template <typename T, int LPR, int GATE>
__global__ void __launch_bounds__(kGnThreads) gated_norm_fwd_kernel(GatedNormParams p) {
  constexpr int d = 8 * LPR, kPer = kGnThreads / LPR;
  const int lane = threadIdx.x % LPR;
  float w[8], o[kGnRows][8], g[kGnRows][8];
  load8(p.weight + 8 * lane, w);
  long long row[kGnRows];
  bool in[kGnRows], valid[kGnRows];
#pragma unroll
  for (int u = 0; u < kGnRows; ++u) {
    row[u] = ((long long)blockIdx.x * kGnRows + u) * kPer + threadIdx.x / LPR;
    in[u] = row[u] < p.rows;
    valid[u] = in[u];
    zero8(o[u]);
    zero8(g[u]);
    if (!in[u]) continue;
    long long tok = 0;
    if (GATE != kGateNone || p.lengths) tok = p.H.div(row[u]);
    valid[u] = token_valid(tok, p.T, p.lengths);
    if (!valid[u]) continue;
    load8(static_cast<const T*>(p.o) + row[u] * d + 8 * lane, o[u]);
    if (GATE != kGateNone)
      load8(static_cast<const T*>(p.gate) + tok * p.gate_stride + (row[u] - tok * p.H.d) * d + 8 * lane, g[u]);
  }
#pragma unroll
  for (int u = 0; u < kGnRows; ++u) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) s += o[u][e] * o[u][e];
    const float r = rsqrtf(lanes_sum<LPR>(s) * (1.f / d) + p.eps);
    if (!in[u]) continue;
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      y[e] = o[u][e] * r * w[e];
      if (GATE != kGateNone) {
        const float sg = sigmoid<T>(g[u][e]);
        y[e] *= GATE == kGateSilu ? g[u][e] * sg : sg;
      }
      if (!valid[u]) y[e] = 0.f;
    }
    store8(static_cast<T*>(p.y) + row[u] * d + 8 * lane, y);
  }
}

// Persistent blocks: a thread keeps its eight columns for all its rows, so the weight's
// gradient is summed in registers, then over the block in shared memory.
template <typename T, int LPR, int GATE>
__global__ void __launch_bounds__(kGnThreads) gated_norm_bwd_kernel(GatedNormParams p) {
  constexpr int d = 8 * LPR, kPer = kGnThreads / LPR;
  const int lane = threadIdx.x % LPR;
  float w[8], dw[8];
  load8(p.weight + 8 * lane, w);
  zero8(dw);
  for (long long base = (long long)blockIdx.x * kPer; base < p.rows; base += (long long)gridDim.x * kPer) {
    const long long row = base + threadIdx.x / LPR;
    const bool in = row < p.rows;
    bool valid = in;
    float o[8], g[8], dy[8];
    zero8(o);
    zero8(g);
    zero8(dy);
    if (in) {
      long long tok = 0;
      if (GATE != kGateNone || p.lengths) tok = p.H.div(row);
      valid = token_valid(tok, p.T, p.lengths);
      if (valid) {
        load8(static_cast<const T*>(p.o) + row * d + 8 * lane, o);
        load8(static_cast<const T*>(p.dy) + row * d + 8 * lane, dy);
        if (GATE != kGateNone)
          load8(static_cast<const T*>(p.gate) + tok * p.gate_stride + (row - tok * p.H.d) * d + 8 * lane, g);
      }
    }
    float s = 0.f, c = 0.f, dg[8], t[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      s += o[e] * o[e];
      t[e] = dy[e];
      if (GATE != kGateNone) {
        const float sg = sigmoid<T>(g[e]);
        const float slope = GATE == kGateSilu ? sg * (1.f + g[e] * (1.f - sg)) : sg * (1.f - sg);
        dg[e] = dy[e] * slope;  // times xh w below
        t[e] *= GATE == kGateSilu ? g[e] * sg : sg;
      }
      c += t[e] * w[e] * o[e];
    }
    const float r = rsqrtf(lanes_sum<LPR>(s) * (1.f / d) + p.eps);
    const float mean = lanes_sum<LPR>(c) * r * (1.f / d);
    if (!in) continue;
    float d_o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float xh = o[e] * r;
      if (valid) dw[e] += t[e] * xh;
      d_o[e] = valid ? r * (t[e] * w[e] - xh * mean) : 0.f;
      if (GATE != kGateNone) dg[e] = valid ? dg[e] * xh * w[e] : 0.f;
    }
    store8(static_cast<T*>(p.y) + row * d + 8 * lane, d_o);
    if (GATE != kGateNone) store8(static_cast<T*>(p.d_gate) + row * d + 8 * lane, dg);
  }
  __shared__ __align__(16) float sum[kPer][d];
  store8(&sum[threadIdx.x / LPR][8 * lane], dw);
  __syncthreads();
  for (int c = threadIdx.x; c < d; c += kGnThreads) {
    float s = 0.f;
    for (int i = 0; i < kPer; ++i) s += sum[i][c];
    p.part[(size_t)blockIdx.x * d + c] = s;
  }
}

// ------------------------------------------------------------------------------ block norm
// A group of tpr threads holds a row, E columns per thread: tpr is a power of two up to 32,
// or a multiple of 32.  VEC: eight consecutive columns per 16-byte access (D a multiple of
// 8); otherwise one column per access, consecutive threads on consecutive columns.
template <bool VEC>
__device__ __forceinline__ int column(int e, int gt, int tpr) {
  return VEC ? (e / 8) * 8 * tpr + 8 * gt + e % 8 : gt + e * tpr;
}

template <int E, bool VEC, typename T>
__device__ __forceinline__ void load_row(const T* p, int gt, int tpr, int D, bool ok, float (&x)[E]) {
#pragma unroll
  for (int e = 0; e < E; e += VEC ? 8 : 1) {
    const int c = column<VEC>(e, gt, tpr);
    if (VEC) {
      float v[8];
      zero8(v);
      if (ok && c < D) load8(p + c, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[(e + i) % E] = v[i];
    } else {
      x[e] = ok && c < D ? load1(p + c) : 0.f;
    }
  }
}

template <int E, bool VEC, typename T>
__device__ __forceinline__ void store_row(T* p, int gt, int tpr, int D, const float (&x)[E]) {
#pragma unroll
  for (int e = 0; e < E; e += VEC ? 8 : 1) {
    const int c = column<VEC>(e, gt, tpr);
    if (c >= D) continue;
    if (VEC) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = x[(e + i) % E];
      store8(p + c, v);
    } else {
      st1<T>(p + c, x[e]);
    }
  }
}

// per-channel vector; `other` where there is none
template <int E, bool VEC>
__device__ __forceinline__ void load_vec(const float* p, int gt, int tpr, int D, float other, float (&x)[E]) {
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int c = column<VEC>(e, gt, tpr);
    x[e] = c < D ? (p ? __ldg(p + c) : other) : 0.f;
  }
}

// Sum of each of the N values over the group, for every thread of it.  Groups of more than
// one warp meet at a named barrier of their own; `buf` alternates between two shared arrays,
// so that one barrier per reduction is enough.
template <int N>
struct GroupSum {
  float (*buf)[2][32][N];  // [group][parity][warp][N]
  int parity = 0;
  __device__ __forceinline__ void run(float (&x)[N], int group, int gt, int tpr) {
    const int width = tpr < 32 ? tpr : 32;
    for (int off = width / 2; off > 0; off >>= 1) {
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] += __shfl_xor_sync(0xffffffffu, x[i], off);
    }
    if (tpr <= 32) return;
    if (gt % 32 == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) buf[group][parity][gt / 32][i] = x[i];
    }
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(tpr) : "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = 0.f;
    for (int w = 0; w < tpr / 32; ++w) {
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] += buf[group][parity][w][i];
    }
    parity ^= 1;
  }
};

constexpr int kBnThreads = 512;  // most threads of a block
constexpr int kBnGroups = 8;     // most groups of more than one warp in a block

template <typename X, typename A, int E, bool VEC, bool DELTA, bool POST>
__global__ void __launch_bounds__(kBnThreads) block_norm_fwd_kernel(BlockNormParams p) {
  constexpr int R = E == 8 ? 2 : 1;  // rows in flight
  __shared__ float buf[kBnGroups][2][32][R];
  const int tpr = p.tpr, gt = threadIdx.x % tpr, group = threadIdx.x / tpr, D = p.D;
  GroupSum<R> sum{buf};
  float w[E], k[E], wp[E];
  load_vec<E, VEC>(p.weight, gt, tpr, D, 1.f, w);
  if (DELTA) {
    load_vec<E, VEC>(p.scale, gt, tpr, D, 1.f, k);
#pragma unroll
    for (int e = 0; e < E; ++e) k[e] *= p.res_scale;
  }
  if (POST) load_vec<E, VEC>(p.post_weight, gt, tpr, D, 1.f, wp);
  const long long per = (long long)p.groups * R;
  for (long long base = blockIdx.x * per; base < p.rows; base += gridDim.x * per) {
    float x[R][E], y[R][E], s[R];
    long long row[R];
    bool in[R], ok[R];
#pragma unroll
    for (int u = 0; u < R; ++u) {
      row[u] = base + (long long)group * R + u;
      in[u] = row[u] < p.rows;
      ok[u] = in[u] && token_valid(row[u], p.T, p.lengths);
      load_row<E, VEC>(static_cast<const X*>(p.x) + row[u] * D, gt, tpr, D, ok[u], x[u]);
      if (DELTA) load_row<E, VEC>(static_cast<const A*>(p.y) + row[u] * D, gt, tpr, D, ok[u], y[u]);
    }
    if (POST) {
#pragma unroll
      for (int u = 0; u < R; ++u) {
        s[u] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s[u] += y[u][e] * y[u][e];
      }
      sum.run(s, group, gt, tpr);
#pragma unroll
      for (int u = 0; u < R; ++u) {
        const float ry = rsqrtf(s[u] / D + p.eps);
#pragma unroll
        for (int e = 0; e < E; ++e) y[u][e] *= ry * wp[e];
      }
    }
#pragma unroll
    for (int u = 0; u < R; ++u) {
      s[u] = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (DELTA) x[u][e] += k[e] * y[u][e];
        s[u] += x[u][e] * x[u][e];
      }
      if (DELTA && in[u]) store_row<E, VEC>(static_cast<X*>(p.x_out) + row[u] * D, gt, tpr, D, x[u]);
    }
    sum.run(s, group, gt, tpr);
#pragma unroll
    for (int u = 0; u < R; ++u) {
      const float r = rsqrtf(s[u] / D + p.eps);
#pragma unroll
      for (int e = 0; e < E; ++e) x[u][e] *= r * w[e];
      if (in[u]) store_row<E, VEC>(static_cast<A*>(p.h) + row[u] * D, gt, tpr, D, x[u]);
    }
  }
}

// SCALE: there is a per-channel scale whose gradient is wanted.
template <typename X, typename A, int E, bool VEC, bool DELTA, bool POST, bool SCALE>
__global__ void __launch_bounds__(kBnThreads) block_norm_bwd_kernel(BlockNormParams p) {
  constexpr bool Y = POST || SCALE;  // whether y is needed
  constexpr int N = POST ? 3 : 2;
  __shared__ float buf[kBnGroups][2][32][N];
  __shared__ float buf1[kBnGroups][2][32][1];
  extern __shared__ float cols[];  // [groups, tpr * E]: the groups' column sums
  const int tpr = p.tpr, gt = threadIdx.x % tpr, group = threadIdx.x / tpr, D = p.D;
  GroupSum<N> sum{buf};
  GroupSum<1> sum1{buf1};
  float w[E], k[E], wp[E], aw[E], ap[E], as[E];
  load_vec<E, VEC>(p.weight, gt, tpr, D, 1.f, w);
  if (DELTA) {
    load_vec<E, VEC>(p.scale, gt, tpr, D, 1.f, k);
#pragma unroll
    for (int e = 0; e < E; ++e) k[e] *= p.res_scale;
  }
  if (POST) load_vec<E, VEC>(p.post_weight, gt, tpr, D, 1.f, wp);
#pragma unroll
  for (int e = 0; e < E; ++e) aw[e] = ap[e] = as[e] = 0.f;
  for (long long base = (long long)blockIdx.x * p.groups; base < p.rows; base += (long long)gridDim.x * p.groups) {
    const long long row = base + group;
    const bool in = row < p.rows, ok = in && token_valid(row, p.T, p.lengths);
    float x[E], dh[E], dx[E], y[E], s[N];
    load_row<E, VEC>(static_cast<const X*>(p.x) + row * D, gt, tpr, D, ok, x);
    load_row<E, VEC>(static_cast<const A*>(p.dh) + row * D, gt, tpr, D, ok, dh);
    load_row<E, VEC>(static_cast<const X*>(p.dx_in) + row * D, gt, tpr, D, ok && p.dx_in, dx);
    if (Y) load_row<E, VEC>(static_cast<const A*>(p.y) + row * D, gt, tpr, D, ok, y);
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      s[0] += x[e] * x[e];
      s[1] += dh[e] * w[e] * x[e];
      if (POST) s[N - 1] += y[e] * y[e];
    }
    sum.run(s, group, gt, tpr);
    const float r = rsqrtf(s[0] / D + p.eps), mean = s[1] * r / D;
    const float ry = POST ? rsqrtf(s[N - 1] / D + p.eps) : 1.f;
    float c[1] = {0.f};
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float xh = x[e] * r;
      if (ok) aw[e] += dh[e] * xh;
      dx[e] += r * (dh[e] * w[e] - xh * mean);
      if (Y) y[e] *= ry;                                            // yh
      if (SCALE && ok) as[e] += dx[e] * (POST ? y[e] * wp[e] : y[e]);  // times res_scale at the end
      if (POST) {
        const float dz = k[e] * dx[e];
        if (ok) ap[e] += dz * y[e];
        c[0] += dz * wp[e] * y[e];
      }
    }
    if (in) store_row<E, VEC>(static_cast<X*>(p.x_out) + row * D, gt, tpr, D, dx);
    if (DELTA) {
      if (POST) sum1.run(c, group, gt, tpr);
      const float my = c[0] / D;
#pragma unroll
      for (int e = 0; e < E; ++e) dx[e] = POST ? ry * (k[e] * dx[e] * wp[e] - y[e] * my) : k[e] * dx[e];
      if (in) store_row<E, VEC>(static_cast<A*>(p.h) + row * D, gt, tpr, D, dx);
    }
  }
  // column sums of the block: one vector after the other through shared memory
  constexpr int kVec = 1 + (POST ? 1 : 0) + (SCALE ? 1 : 0);
#pragma unroll
  for (int v = 0; v < kVec; ++v) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float a = v == 0 ? aw[e] : (POST && v == 1 ? ap[e] : as[e] * p.res_scale);
      cols[group * tpr * E + column<VEC>(e, gt, tpr)] = a;
    }
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += blockDim.x) {
      float t = 0.f;
      for (int g = 0; g < p.groups; ++g) t += cols[g * tpr * E + c];
      p.part[((size_t)blockIdx.x * kVec + v) * D + c] = t;
    }
  }
}

constexpr int kSumCols = 32, kSumSlices = 32;

__global__ void __launch_bounds__(kSumCols * kSumSlices) column_sum_kernel(ColumnSumParams p) {
  __shared__ float sm[kSumSlices][kSumCols + 1];
  const int col = blockIdx.x * kSumCols + threadIdx.x % kSumCols, slice = threadIdx.x / kSumCols;
  const int n = p.nvec * p.D;
  float s = 0.f;
  if (col < n)
    for (int b = slice; b < p.blocks; b += kSumSlices) s += p.part[(size_t)b * n + col];
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

template <typename T, int LPR>
cudaError_t gated_fwd_lanes(const GatedNormParams& p, int gate, cudaStream_t stream) {
  const long long per = (long long)kGnRows * (kGnThreads / LPR);
  const long long blocks = (p.rows + per - 1) / per;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  if (gate == kGateNone)
    gated_norm_fwd_kernel<T, LPR, kGateNone><<<(int)blocks, kGnThreads, 0, stream>>>(p);
  else if (gate == kGateSilu)
    gated_norm_fwd_kernel<T, LPR, kGateSilu><<<(int)blocks, kGnThreads, 0, stream>>>(p);
  else
    gated_norm_fwd_kernel<T, LPR, kGateSigmoid><<<(int)blocks, kGnThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

template <typename T, int LPR>
cudaError_t gated_bwd_lanes(const GatedNormParams& p, int gate, int blocks, cudaStream_t stream) {
  if (gate == kGateNone)
    gated_norm_bwd_kernel<T, LPR, kGateNone><<<blocks, kGnThreads, 0, stream>>>(p);
  else if (gate == kGateSilu)
    gated_norm_bwd_kernel<T, LPR, kGateSilu><<<blocks, kGnThreads, 0, stream>>>(p);
  else
    gated_norm_bwd_kernel<T, LPR, kGateSigmoid><<<blocks, kGnThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

// Threads per row and rows per block of the block norm.
void block_norm_shape(int D, int* tpr, int* groups, int* cols_per_thread) {
  const int E = D <= 8 * kBnThreads ? 8 : 16;
  int t = (D + E - 1) / E;
  if (t <= 32) {
    int q = 1;
    while (q < t) q *= 2;
    *tpr = q;
    *groups = 128 / q;
  } else {
    t = (t + 31) / 32 * 32;
    *tpr = t;
    *groups = t >= 256 ? 1 : 384 / t;
  }
  *cols_per_thread = E;
}

template <typename X, typename A, int E, bool VEC>
cudaError_t block_fwd_cols(const BlockNormParams& p, int blocks, cudaStream_t stream) {
  const int threads = p.tpr * p.groups;
  if (!p.y)
    block_norm_fwd_kernel<X, A, E, VEC, false, false><<<blocks, threads, 0, stream>>>(p);
  else if (!p.post_weight)
    block_norm_fwd_kernel<X, A, E, VEC, true, false><<<blocks, threads, 0, stream>>>(p);
  else
    block_norm_fwd_kernel<X, A, E, VEC, true, true><<<blocks, threads, 0, stream>>>(p);
  return cudaGetLastError();
}

template <typename X, typename A, int E, bool VEC>
cudaError_t block_bwd_cols(const BlockNormParams& p, int blocks, cudaStream_t stream) {
  const int threads = p.tpr * p.groups;
  const size_t smem = (size_t)threads * E * sizeof(float);
  if (!p.y)
    block_norm_bwd_kernel<X, A, E, VEC, false, false, false><<<blocks, threads, smem, stream>>>(p);
  else if (!p.post_weight && !p.scale)
    block_norm_bwd_kernel<X, A, E, VEC, true, false, false><<<blocks, threads, smem, stream>>>(p);
  else if (!p.post_weight)
    block_norm_bwd_kernel<X, A, E, VEC, true, false, true><<<blocks, threads, smem, stream>>>(p);
  else if (!p.scale)
    block_norm_bwd_kernel<X, A, E, VEC, true, true, false><<<blocks, threads, smem, stream>>>(p);
  else
    block_norm_bwd_kernel<X, A, E, VEC, true, true, true><<<blocks, threads, smem, stream>>>(p);
  return cudaGetLastError();
}

template <typename X, typename A>
cudaError_t block_norm_types(BlockNormParams p, bool bwd, cudaStream_t stream) {
  int E;
  block_norm_shape(p.D, &p.tpr, &p.groups, &E);
  const int blocks = block_norm_blocks(p.rows, p.D, bwd);
  const bool vec = p.D % 8 == 0;
  if (bwd) {
    if (E == 8) return vec ? block_bwd_cols<X, A, 8, true>(p, blocks, stream) : block_bwd_cols<X, A, 8, false>(p, blocks, stream);
    return vec ? block_bwd_cols<X, A, 16, true>(p, blocks, stream) : block_bwd_cols<X, A, 16, false>(p, blocks, stream);
  }
  if (E == 8) return vec ? block_fwd_cols<X, A, 8, true>(p, blocks, stream) : block_fwd_cols<X, A, 8, false>(p, blocks, stream);
  return vec ? block_fwd_cols<X, A, 16, true>(p, blocks, stream) : block_fwd_cols<X, A, 16, false>(p, blocks, stream);
}

}  // namespace

int block_norm_blocks(long long rows, int D, bool bwd) {
  int tpr, groups, E;
  block_norm_shape(D, &tpr, &groups, &E);
  const long long per = (long long)groups * (!bwd && E == 8 ? 2 : 1);
  const int threads = tpr * groups, fill = bwd ? 768 : 1536;
  const long long need = (rows + per - 1) / per, most = (long long)kSMs * (threads < fill ? fill / threads : 1);
  return (int)(need < most ? need : most);
}

cudaError_t launch_column_sum(const ColumnSumParams& p, cudaStream_t stream) {
  const int cols = p.nvec * p.D;
  column_sum_kernel<<<(cols + kSumCols - 1) / kSumCols, kSumCols * kSumSlices, 0, stream>>>(p);
  return cudaGetLastError();
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

// d_weight [d] is the sum of the blocks' partial sums.
cudaError_t launch_gated_norm_bwd(const GatedNormParams& p, int d, int gate, int dtype, float* d_weight,
                                  cudaStream_t stream) {
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
  if (err != cudaSuccess) return err;
  ColumnSumParams c{p.part, {d_weight, nullptr, nullptr}, blocks, 1, d};
  return launch_column_sum(c, stream);
}

cudaError_t launch_block_norm(const BlockNormParams& p, bool bwd, int x_dtype, int dtype, float* const (&sums)[3],
                              cudaStream_t stream) {
  cudaError_t err;
  if (x_dtype == PRISM_BF16)
    err = block_norm_types<__nv_bfloat16, __nv_bfloat16>(p, bwd, stream);
  else if (dtype == PRISM_BF16)
    err = block_norm_types<float, __nv_bfloat16>(p, bwd, stream);
  else
    err = block_norm_types<float, float>(p, bwd, stream);
  if (err != cudaSuccess || !bwd) return err;
  ColumnSumParams c{p.part, {sums[0], nullptr, nullptr}, block_norm_blocks(p.rows, p.D, true), 1, p.D};
  if (p.y && p.post_weight) c.out[c.nvec++] = sums[1];
  if (p.y && p.scale) c.out[c.nvec++] = sums[2];
  return launch_column_sum(c, stream);
}

}  // namespace prism
