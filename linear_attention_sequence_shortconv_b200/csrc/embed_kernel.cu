// Embedding lookup and its gradient.
//
//   forward    out[n] = scale * table[ids[n]]
//   backward   d_table[v] (+)= scale * sum over {n : ids[n] = v} of d_out[n]
//
// Tokens of padding (t >= lengths[b]) are not read: their output row is zero and they give no
// gradient.  So is an id outside [0, V), which is recorded in the status word as well.
//
// Backward: the tokens are sorted by id (a stable radix sort of (id, token) pairs, two or
// three passes of up to ten bits), so that a table row's summands stand next to each other in
// the order of the tokens.  Then one launch sums the runs: the sorted positions are cut into
// chunks of equal length, each thread group walks one chunk with its columns in registers and
// writes every run that lies inside the chunk; a run that crosses a chunk's border leaves
// partial sums, which a last launch adds from left to right.  No floating-point atomics, so
// the result does not depend on any order of execution.  Rows without a token are written as
// zero by further blocks of the summing launch, so a dense gradient is written exactly once.
//
// Bound by memory: d_out is read once and the table's gradient is written once; the pairs are
// 8 bytes a token and pass.
#include "embed.cuh"
#include "rowops.cuh"

namespace prism {

namespace {

constexpr int kFwdThreads = 256;

// One id; `key` of a token that takes no part is V.
template <typename I>
__device__ __forceinline__ uint32_t token_key(const EmbedParams& p, long long n, bool small) {
  if (!token_valid(n, p.T, p.lengths, small)) return (uint32_t)p.V;
  const long long id = static_cast<const I*>(p.ids)[n];
  if (id >= 0 && id < p.V) return (uint32_t)id;
  record_status(p.status, PRISM_ERR_BOUNDS);
  return (uint32_t)p.V;
}

// A block takes `tile` tokens: their keys go to shared memory, then its threads walk the rows'
// 16-byte (eight-element) pieces one after the other, so that no lane idles at any width.
template <typename I, typename W, typename T, bool VEC>
__global__ void __launch_bounds__(kFwdThreads) embed_fwd_kernel(EmbedParams p, int tile, int pieces) {
  __shared__ uint32_t key[kEmbedFwdTile];
  const long long first = (long long)blockIdx.x * tile;
  const int rows = (int)(p.N - first < tile ? p.N - first : tile);
  for (int i = threadIdx.x; i < rows; i += kFwdThreads) key[i] = token_key<I>(p, first + i, true);
  __syncthreads();
  const W* table = static_cast<const W*>(p.table);
  T* out = static_cast<T*>(p.out) + first * p.D;
  const int n = rows * pieces;
#pragma unroll 4
  for (int i = threadIdx.x; i < n; i += kFwdThreads) {
    const int r = (int)((uint32_t)i / (uint32_t)pieces), c = i - r * pieces;
    const bool ok = key[r] < (uint32_t)p.V;
    if (VEC) {
      float x[8];
      zero8(x);
      if (ok) load8(table + (size_t)key[r] * p.D + 8 * c, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= p.scale;
      store8(out + (size_t)r * p.D + 8 * c, x);
    } else {
      st1<T>(out + (size_t)r * p.D + c, ok ? load1(table + (size_t)key[r] * p.D + c) * p.scale : 0.f);
    }
  }
}

// ------------------------------------------------------------------------------------ the sort
constexpr int kSortThreads = 512, kSortWarps = kSortThreads / 32;
constexpr int kMaxBins = 1 << kEmbedMaxDigit;
constexpr uint32_t kNoKey = 0xffffffffu;  // a place behind the tile's last token

// Counts of the first digit per tile; clears the later digits' counts of this tile.
template <typename I>
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(EmbedParams p, EmbedPlan plan) {
  __shared__ int count[kMaxBins];
  const int bins = 1 << plan.digit;
  for (int i = threadIdx.x; i < bins; i += kSortThreads) count[i] = 0;
  __syncthreads();
  const long long first = (long long)blockIdx.x * plan.tile;
  const long long last = first + plan.tile < p.N ? first + plan.tile : p.N;
  for (long long n = first + threadIdx.x; n < last; n += kSortThreads)
    atomicAdd(&count[token_key<I>(p, n, true) & (bins - 1)], 1);
  __syncthreads();
  for (int i = threadIdx.x; i < bins; i += kSortThreads) {
    p.hist[(size_t)blockIdx.x * bins + i] = count[i];
    for (int q = 1; q < plan.passes; ++q) p.hist[((size_t)q * plan.tiles + blockIdx.x) * bins + i] = 0;
  }
}

// One pass: a tile's pairs move to their places for digit `pass`.  Every block adds up the
// counts of all tiles itself (they are few, and stay in L2).  Within a tile the warps take
// consecutive runs of 32 * ROUNDS pairs; a pair's rank is the number of equal digits before
// it, counted per warp, then over the warps.  The next digit's counts are gathered on the
// way (integers, so their order does not matter).
template <typename I, int ROUNDS>
__global__ void __launch_bounds__(kSortThreads) sort_pass_kernel(EmbedParams p, EmbedPlan plan, int pass) {
  __shared__ unsigned short warp_count[kSortWarps][kMaxBins];
  __shared__ int base[kMaxBins], step[kMaxBins];
  __shared__ int warp_total[kSortWarps];
  const int bins = 1 << plan.digit, shift = pass * plan.digit;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int* hist = p.hist + (size_t)pass * plan.tiles * bins;
  int* next = pass + 1 < plan.passes ? p.hist + (size_t)(pass + 1) * plan.tiles * bins : nullptr;
  const uint32_t* key_in = pass ? p.keys[(pass - 1) & 1] : nullptr;
  const uint32_t* tok_in = pass ? p.toks[(pass - 1) & 1] : nullptr;
  uint32_t* key_out = p.keys[pass & 1];
  uint32_t* tok_out = p.toks[pass & 1];

  // base[b] = pairs with a smaller digit + pairs of digit b in earlier tiles
  int total[kMaxBins / kSortThreads], before[kMaxBins / kSortThreads], sum = 0;
#pragma unroll
  for (int j = 0; j < kMaxBins / kSortThreads; ++j) {
    // consecutive bins per thread, so that one scan over the threads orders all bins
    const int b = threadIdx.x * (kMaxBins / kSortThreads) + j;
    total[j] = before[j] = 0;
    if (b < bins) {
#pragma unroll 8
      for (int t = 0; t < plan.tiles; ++t) {
        const int c = hist[(size_t)t * bins + b];
        total[j] += c;
        if (t < (int)blockIdx.x) before[j] += c;
      }
    }
    sum += total[j];
  }
  int scan = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, scan, off);
    if (lane >= off) scan += y;
  }
  if (lane == 31) warp_total[warp] = scan;
  __syncthreads();
  int run = scan - sum;
  for (int w = 0; w < warp; ++w) run += warp_total[w];
#pragma unroll
  for (int j = 0; j < kMaxBins / kSortThreads; ++j) {
    const int b = threadIdx.x * (kMaxBins / kSortThreads) + j;
    if (b < bins) base[b] = run + before[j];
    run += total[j];
  }

  const long long first = (long long)blockIdx.x * plan.tile;
  const long long last = first + plan.tile < p.N ? first + plan.tile : p.N;
  for (int b = threadIdx.x; b < bins; b += kSortThreads) step[b] = 0;
  __syncthreads();
  for (long long sub = first; sub < last; sub += kSortThreads * ROUNDS) {
    for (int b = threadIdx.x; b < bins; b += kSortThreads) base[b] += step[b];
    for (int i = threadIdx.x; i < kSortWarps * bins; i += kSortThreads) warp_count[i >> plan.digit][i & (bins - 1)] = 0;
    __syncthreads();
    uint32_t key[ROUNDS], tok[ROUNDS];
    int rank[ROUNDS];
#pragma unroll
    for (int i = 0; i < ROUNDS; ++i) {
      const long long n = sub + (long long)warp * 32 * ROUNDS + 32 * i + lane;
      key[i] = kNoKey;
      tok[i] = 0;
      if (n < last) {
        key[i] = pass ? key_in[n] : token_key<I>(p, n, true);
        tok[i] = pass ? tok_in[n] : (uint32_t)n;
      }
    }
#pragma unroll
    for (int i = 0; i < ROUNDS; ++i) {
      const bool in = key[i] != kNoKey;
      const uint32_t digit = in ? (key[i] >> shift) & (bins - 1) : kNoKey;
      const uint32_t same = __match_any_sync(0xffffffffu, digit);
      const int leader = __ffs(same) - 1;
      int start = 0;
      if (in && lane == leader) {
        start = warp_count[warp][digit];
        warp_count[warp][digit] = (unsigned short)(start + __popc(same));
      }
      rank[i] = __shfl_sync(0xffffffffu, start, leader) + __popc(same & ((1u << lane) - 1));
      __syncwarp();
    }
    __syncthreads();
    for (int b = threadIdx.x; b < bins; b += kSortThreads) {
      int s = 0;
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) {
        const int c = warp_count[w][b];
        warp_count[w][b] = (unsigned short)s;
        s += c;
      }
      step[b] = s;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ROUNDS; ++i) {
      if (key[i] == kNoKey) continue;
      const uint32_t digit = (key[i] >> shift) & (bins - 1);
      const int at = base[digit] + warp_count[warp][digit] + rank[i];
      if (!in_bounds(at, p.N, p.status)) continue;
      key_out[at] = key[i];
      tok_out[at] = tok[i];
      if (next) atomicAdd(next + (size_t)(at / plan.tile) * bins + ((key[i] >> (shift + plan.digit)) & (bins - 1)), 1);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------------------------ the sums
// Eight columns per thread: consecutive ones where D is a multiple of 8, else one of every
// tpr.  blockIdx.y is the tile of 8 tpr columns.
constexpr int kSumThreads = 256;
constexpr int kZeroRows = 64;  // table rows that one zeroing block looks after
constexpr int kAhead = 4;      // rows in flight per thread

template <bool VEC>
struct Columns {
  int first, step, D;  // column of element e: first + e * step
  __device__ __forceinline__ Columns(int gt, int tpr, int tile, int D_)
      : first(tile * 8 * tpr + (VEC ? 8 * gt : gt)), step(VEC ? 1 : tpr), D(D_) {}
  template <typename T>
  __device__ __forceinline__ void load(const T* row, float (&x)[8]) const {
    zero8(x);
    if (VEC) {
      if (first < D) load8(row + first, x);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (first + e * step < D) x[e] = load1(row + first + e * step);
    }
  }
  __device__ __forceinline__ void store(float* row, const float (&x)[8]) const {
    if (VEC) {
      if (first < D) store8(row + first, x);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (first + e * step < D) row[first + e * step] = x[e];
    }
  }
  // the finished sum of table row v
  __device__ __forceinline__ void finish(const EmbedParams& p, uint32_t v, const float (&x)[8]) const {
    float* row = p.d_table + (size_t)v * D;
    float y[8];
    if (p.accumulate) load(row, y);
    else zero8(y);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] += p.scale * x[e];
    store(row, y);
  }
};

// first position in [0, N) whose key is at least v
__device__ __forceinline__ int lower_bound(const uint32_t* keys, int N, uint32_t v) {
  int lo = 0, hi = N;
  while (lo < hi) {
    const int mid = lo + (hi - lo) / 2;
    if (keys[mid] < v) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

// table rows [v0, v0 + kZeroRows): those without a token become zero
__device__ __forceinline__ void zero_absent_rows(const EmbedParams& p, const uint32_t* keys, long long v0) {
  __shared__ int range[2];
  __shared__ int present[kZeroRows];
  const int rows = (int)(p.V - v0 < kZeroRows ? p.V - v0 : kZeroRows);
  if (threadIdx.x < 2) range[threadIdx.x] = lower_bound(keys, (int)p.N, (uint32_t)(v0 + (threadIdx.x ? rows : 0)));
  if (threadIdx.x < kZeroRows) present[threadIdx.x] = 0;
  __syncthreads();
  for (int i = range[0] + threadIdx.x; i < range[1]; i += blockDim.x) present[keys[i] - (uint32_t)v0] = 1;
  __syncthreads();
  const float zero[8] = {};
  const bool vec = p.D % 8 == 0;
  const int pieces = vec ? p.D / 8 : p.D;
  for (int r = 0; r < rows; ++r) {
    if (present[r]) continue;
    float* row = p.d_table + (size_t)(v0 + r) * p.D;
    for (int c = threadIdx.x; c < pieces; c += blockDim.x) {
      if (vec) store8(row + 8 * c, zero);
      else row[c] = 0.f;
    }
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kSumThreads) embed_sum_kernel(EmbedParams p, EmbedPlan plan, int tpr, int groups,
                                                                int sum_blocks) {
  const uint32_t* keys = p.keys[(plan.passes - 1) & 1];
  const uint32_t* toks = p.toks[(plan.passes - 1) & 1];
  if ((int)blockIdx.x >= sum_blocks) {
    if (blockIdx.y == 0) zero_absent_rows(p, keys, (long long)(blockIdx.x - sum_blocks) * kZeroRows);
    return;
  }
  const int group = threadIdx.x / tpr;
  const long long c = (long long)blockIdx.x * groups + group;
  if (c >= plan.chunks) return;
  const int s = (int)c * plan.chunk, e = (int)(s + (long long)plan.chunk < p.N ? s + plan.chunk : p.N);
  const Columns<VEC> col(threadIdx.x - group * tpr, tpr, blockIdx.y, p.D);
  const uint32_t none = (uint32_t)p.V;
  uint32_t cur = keys[s];
  if (cur == none) return;  // padding sorts behind every id
  const T* d_out = static_cast<const T*>(p.d_out);
  float* head = p.part + (size_t)c * 2 * p.D;
  bool from_before = s > 0 && keys[s - 1] == cur;
  float acc[8];
  zero8(acc);
  for (int i = s; i < e; i += kAhead) {
    uint32_t key[kAhead];
    float x[kAhead][8];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      key[j] = i + j < e ? keys[i + j] : none;
      if (key[j] != none) col.load(d_out + (size_t)toks[i + j] * p.D, x[j]);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (i + j >= e) break;
      if (key[j] != cur) {
        if (from_before) col.store(head, acc);
        else col.finish(p, cur, acc);
        from_before = false;
        cur = key[j];
        if (cur == none) return;
        zero8(acc);
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) acc[q] += x[j][q];
    }
  }
  const bool goes_on = e < p.N && keys[e] == cur;
  if (from_before) col.store(head, acc);
  else if (goes_on) col.store(head + p.D, acc);  // this chunk's tail
  else col.finish(p, cur, acc);
}

// The runs that cross a chunk's border: the group of the chunk where a run begins adds the
// chunk's tail and the heads of the chunks it reaches, from left to right.
template <bool VEC>
__global__ void __launch_bounds__(kSumThreads) embed_join_kernel(EmbedParams p, EmbedPlan plan, int tpr, int groups) {
  const uint32_t* keys = p.keys[(plan.passes - 1) & 1];
  const int group = threadIdx.x / tpr;
  const long long c = (long long)blockIdx.x * groups + group;
  if (c + 1 >= plan.chunks) return;
  const int s = (int)c * plan.chunk, e = s + plan.chunk;  // not the last chunk: e < N
  const uint32_t cur = keys[e - 1];
  if (cur == (uint32_t)p.V || keys[e] != cur) return;
  if (s > 0 && keys[s - 1] == cur) return;  // began earlier (the keys are sorted)
  const Columns<VEC> col(threadIdx.x - group * tpr, tpr, blockIdx.y, p.D);
  float acc[8], x[8];
  col.load(p.part + ((size_t)c * 2 + 1) * p.D, acc);
  for (long long n = c + 1; n < plan.chunks && keys[n * plan.chunk] == cur; ++n) {
    col.load(p.part + (size_t)n * 2 * p.D, x);
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[q] += x[q];
  }
  col.finish(p, cur, acc);
}

template <typename I, typename W, typename T>
cudaError_t embed_fwd_types(const EmbedParams& p, cudaStream_t stream) {
  const bool vec = p.D % 8 == 0;
  const int pieces = vec ? p.D / 8 : p.D;
  // about eight pieces per thread and block
  int tile = 8 * kFwdThreads / pieces;
  tile = tile < 1 ? 1 : tile > kEmbedFwdTile ? kEmbedFwdTile : tile;
  const int blocks = (int)((p.N + tile - 1) / tile);
  if (vec)
    embed_fwd_kernel<I, W, T, true><<<blocks, kFwdThreads, 0, stream>>>(p, tile, pieces);
  else
    embed_fwd_kernel<I, W, T, false><<<blocks, kFwdThreads, 0, stream>>>(p, tile, pieces);
  return cudaGetLastError();
}

template <typename I>
cudaError_t embed_fwd_ids(const EmbedParams& p, int table_dtype, int dtype, cudaStream_t stream) {
  if (table_dtype == PRISM_BF16) return embed_fwd_types<I, __nv_bfloat16, __nv_bfloat16>(p, stream);
  if (dtype == PRISM_BF16) return embed_fwd_types<I, float, __nv_bfloat16>(p, stream);
  return embed_fwd_types<I, float, float>(p, stream);
}

template <typename I>
cudaError_t embed_sort(const EmbedParams& p, const EmbedPlan& plan, cudaStream_t stream) {
  sort_count_kernel<I><<<plan.tiles, kSortThreads, 0, stream>>>(p, plan);
  for (int pass = 0; pass < plan.passes; ++pass) {
    if (plan.rounds == 2)
      sort_pass_kernel<I, 2><<<plan.tiles, kSortThreads, 0, stream>>>(p, plan, pass);
    else
      sort_pass_kernel<I, 8><<<plan.tiles, kSortThreads, 0, stream>>>(p, plan, pass);
  }
  return cudaGetLastError();
}

template <typename T, bool VEC>
cudaError_t embed_sums(const EmbedParams& p, const EmbedPlan& plan, cudaStream_t stream) {
  const int need = (p.D + 7) / 8;  // threads that hold a row
  int tpr = need < kSumThreads ? need : kSumThreads;
  const int groups = kSumThreads / tpr, tiles = (need + tpr - 1) / tpr;
  const int sum_blocks = (plan.chunks + groups - 1) / groups;
  const int zero_blocks = p.accumulate ? 0 : (int)(((long long)p.V + kZeroRows - 1) / kZeroRows);
  embed_sum_kernel<T, VEC><<<dim3(sum_blocks + zero_blocks, tiles), tpr * groups, 0, stream>>>(p, plan, tpr, groups,
                                                                                              sum_blocks);
  if (plan.chunks > 1)
    embed_join_kernel<VEC><<<dim3(sum_blocks, tiles), tpr * groups, 0, stream>>>(p, plan, tpr, groups);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_embed_fwd(const EmbedParams& p, int ids_bits, int table_dtype, int dtype, cudaStream_t stream) {
  return ids_bits == 32 ? embed_fwd_ids<int32_t>(p, table_dtype, dtype, stream)
                        : embed_fwd_ids<long long>(p, table_dtype, dtype, stream);
}

cudaError_t launch_embed_bwd(const EmbedParams& p, int ids_bits, int dtype, cudaStream_t stream) {
  const EmbedPlan plan(p.N, p.V, p.D);
  const cudaError_t err = ids_bits == 32 ? embed_sort<int32_t>(p, plan, stream) : embed_sort<long long>(p, plan, stream);
  if (err != cudaSuccess) return err;
  const bool vec = p.D % 8 == 0;
  if (dtype == PRISM_FP32)
    return vec ? embed_sums<float, true>(p, plan, stream) : embed_sums<float, false>(p, plan, stream);
  return vec ? embed_sums<__nv_bfloat16, true>(p, plan, stream) : embed_sums<__nv_bfloat16, false>(p, plan, stream);
}

}  // namespace prism
