// Embedding lookup and its gradient.
//
//   forward    out[n] = scale * table[ids[n]]
//   backward   d_table[v] (+)= scale * sum over {n : ids[n] = v} of d_out[n]
//
// Tokens of padding (t >= lengths[b]) are not read: their output row is zero and they give no
// gradient.  So is an id outside [0, V), which is recorded in the status word as well.
//
// Backward: the tokens are sorted by id (a stable radix sort of (id, token) pairs in passes of
// up to ten bits), so that a table row's summands stand next to each other in the order of
// the tokens.  Then one launch sums the runs: the sorted positions are cut into chunks of
// equal length, each thread group walks one chunk with its columns in registers and writes
// every run that lies inside the chunk; a run that crosses a chunk's border leaves partial
// sums, which a last launch adds in a fixed order.  No floating-point atomics, so the result
// does not depend on any order of execution.  Very many chunks have the partial sums of long runs
// folded in between.  Rows without a token (a bitmap that the sort leaves) are written as zero
// by further blocks of the summing launch, so a dense gradient is written exactly once.
//
// The lookup is bound by memory (recommendation batch, 128 x 1024 ragged tokens, a table of
// 1000003 x 128 in fp32: 12 us, 4.1 TB/s).  The gradient reads d_out once and writes the table's
// gradient once, but about half of its time is a chain of steps that each wait for the one
// before: with rows of 8 elements, where there is nothing to move, 32768 tokens take 33 us (sort
// 13.5, sums 14, joins 8, less what the chained launches overlap).  Measured: 130M LM, 32768
// tokens, dense gradient of 32000 x 768: 56 us (floor 22.7); recommendation batch, added to
// 1000003 x 128: 51 us (floor 11); a million tokens over two rows of 64: 71 us (without the
// fold 1154), over 3000: 118 us (searching the sorted keys for rows without a token: 205).
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>

#include "embed.cuh"
#include "rowops.cuh"

namespace prism {

namespace {

std::atomic<bool> g_portable_clusters{false};  // prism_set_portable_clusters()

constexpr int kFwdThreads = 256;

// One id; `key` of a token that takes no part is V.
template <typename I>
__device__ __forceinline__ uint32_t token_key(const EmbedParams& p, long long n) {
  if (!token_valid(n, p.T, p.lengths)) return (uint32_t)p.V;
  const long long id = static_cast<const I*>(p.ids)[n];
  if (id >= 0 && id < p.V) return (uint32_t)id;
  record_status(p.status, PRISM_ERR_BOUNDS);
  return (uint32_t)p.V;
}

// A block takes `tile` tokens: their keys go to shared memory, then its threads walk the rows'
// 16-byte (eight-element) pieces one after the other, so that no lane idles at any width.
template <typename I, typename W, typename T, bool VEC>
__global__ void __launch_bounds__(kFwdThreads) embed_fwd_kernel(EmbedParams p, int tile, FastDiv pieces) {
  __shared__ uint32_t key[kEmbedFwdTile];
  const long long first = (long long)blockIdx.x * tile;
  const int rows = (int)(p.N - first < tile ? p.N - first : tile);
  for (int i = threadIdx.x; i < rows; i += kFwdThreads) key[i] = token_key<I>(p, first + i);
  __syncthreads();
  const W* table = static_cast<const W*>(p.table);
  T* out = static_cast<T*>(p.out) + first * p.D;
  const int n = rows * (int)pieces.d;
#pragma unroll 4
  for (int i = threadIdx.x; i < n; i += kFwdThreads) {
    const int r = (int)pieces.div32((uint32_t)i), c = i - r * (int)pieces.d;
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
constexpr int kMaxBins = 1 << kEmbedMaxDigit;
constexpr uint32_t kNoKey = 0xffffffffu;  // a place behind the last token

// The bits of the table rows that a token names (dense gradients only): cleared by the first
// sorting launch, set once per block or run.
__device__ __forceinline__ void clear_present(const EmbedParams& p, int block, int blocks) {
  if (!p.present) return;
  const int pieces = (int)(((long long)p.V + 127) / 128);  // of 16 bytes, as the bitmap's room is
  for (int i = block * blockDim.x + threadIdx.x; i < pieces; i += blocks * blockDim.x)
    reinterpret_cast<uint4*>(p.present)[i] = make_uint4(0, 0, 0, 0);
}
__device__ __forceinline__ void set_present(const EmbedParams& p, uint32_t key) {
  if (p.present && key < (uint32_t)p.V) atomicOr(p.present + key / 32, 1u << key % 32);
}

// Stable ranks of a warp's 32 * KPT consecutive keys among the equal digits of the warp, and
// the warp's counts per digit (`count`, zero before).  The lanes of equal digit are found by one
// vote per bit.
template <int KPT>
__device__ __forceinline__ void rank_in_warp(const uint32_t (&key)[KPT], int shift, int bits, int lane,
                                             unsigned short* count, int (&rank)[KPT]) {
#pragma unroll
  for (int i = 0; i < KPT; ++i) {
    const bool in = key[i] != kNoKey;
    const uint32_t digit = (key[i] >> shift) & ((1u << bits) - 1);
    uint32_t same = __ballot_sync(0xffffffffu, in);
    if (!in) same = ~same;
#pragma unroll
    for (int b = 0; b < kEmbedMaxDigit; ++b) {
      if (b >= bits) break;  // the same for all lanes
      const bool bit = (digit >> b) & 1;
      const uint32_t set = __ballot_sync(0xffffffffu, bit);
      same &= bit ? set : ~set;
    }
    const int leader = __ffs(same) - 1;
    int start = 0;
    if (in && lane == leader) {
      start = count[digit];
      count[digit] = (unsigned short)(start + __popc(same));
    }
    rank[i] = __shfl_sync(0xffffffffu, start, leader) + __popc(same & ((1u << lane) - 1));
    __syncwarp();
  }
}

// The warps' counts of digit b become their exclusive prefix over the warps; returns the sum.
template <int WARPS>
__device__ __forceinline__ int prefix_over_warps(unsigned short* count, int stride, int b) {
  int c[WARPS], s = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) c[w] = count[w * stride + b];
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    count[w * stride + b] = (unsigned short)s;
    s += c[w];
  }
  return s;
}

// The cluster's barrier in its two halves; what a thread wrote before arriving is seen by the
// whole cluster after the wait.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Exclusive scan of one value per thread over a block of `warps` warps (warp_total: shared).
__device__ __forceinline__ int block_exclusive_scan(int x, int warps, int* warp_total) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  int scan = x;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, scan, off);
    if (lane >= off) scan += y;
  }
  if (lane == 31) warp_total[warp] = scan;
  __syncthreads();
  if (warp == 0) {
    int t = lane < warps ? warp_total[lane] : 0;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, t, off);
      if (lane >= off) t += y;
    }
    if (lane < warps) warp_total[lane] = t;
  }
  __syncthreads();
  return scan - x + (warp ? warp_total[warp - 1] : 0);
}

// Up to 1024 * KPT * (cluster size) tokens: the whole sort in one launch of one cluster.  In a
// pass a block ranks its pairs, exchanges its counts per digit with the other blocks through
// distributed shared memory, orders the pairs by digit in its shared memory and writes them
// out from there, so that the pairs of a digit leave in runs.  The cluster's barrier orders a
// pass's pairs before the next one's reads.
//
// Against tiles over all SMs: 32768 tokens 14.5 us here and 26 us by tiles; 131072 tokens 41 us
// (eight pairs a thread, bound by the instructions of 16 SMs) and 26 us.  Of the whole gradient, whose
// chained launches overlap: two passes, 8193 tokens 35.1 us here and 41.0 by tiles, 32768 tokens 38.9
// and 41.8; one pass 33.2 and 32.1, three passes 48.4 and 45.1 at 32768.
constexpr int kClusterThreads = 1024, kClusterWarps = kClusterThreads / 32;

template <typename I, int KPT>
__global__ void __launch_bounds__(kClusterThreads) sort_cluster_kernel(EmbedParams p, EmbedPlan plan) {
  extern __shared__ __align__(16) char sort_smem[];
  const int bins = 1 << plan.digit;
  uint2* staged = reinterpret_cast<uint2*>(sort_smem);                      // [1024 KPT] pairs by digit
  int* total = reinterpret_cast<int*>(staged + kClusterThreads * KPT);      // [bins] this block's counts
  int* local = total + bins;                                                // [bins] first staged place
  int* base = local + bins;                                                 // [bins] first place in the output
  unsigned short* count = reinterpret_cast<unsigned short*>(base + bins);   // [warps][bins]
  __shared__ int warp_total[2][kClusterWarps];
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  const int blocks = (int)cluster.num_blocks(), me = (int)cluster.block_rank();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const long long block0 = (long long)me * kClusterThreads * KPT, first = block0 + warp * 32 * KPT + lane;
  const int mine = (int)(p.N - block0 < kClusterThreads * KPT ? (p.N > block0 ? p.N - block0 : 0) : kClusterThreads * KPT);
  launch_dependents();
  clear_present(p, me, blocks);
  for (int pass = 0; pass < plan.passes; ++pass) {
    const int shift = pass * plan.digit;
    const uint2* in = pass & 1 ? p.pairs[0] : p.pairs[1];
    uint32_t key[KPT], tok[KPT];
    int rank[KPT];
#pragma unroll
    for (int i = 0; i < KPT; ++i) {
      const long long n = first + 32 * i;
      key[i] = kNoKey;
      tok[i] = (uint32_t)n;
      if (n < p.N) {
        if (pass) {  // the pairs of an earlier pass come from other SMs: not through this one's L1
          const uint2 x = __ldcg(in + n);
          key[i] = x.x;
          tok[i] = x.y;
        } else {
          key[i] = token_key<I>(p, n);
        }
      }
    }
    uint32_t* zero = reinterpret_cast<uint32_t*>(count);
    for (int i = threadIdx.x; i < kClusterWarps * bins / 2; i += kClusterThreads) zero[i] = 0;
    __syncthreads();
    rank_in_warp<KPT>(key, shift, plan.digit, lane, count + warp * bins, rank);
    __syncthreads();
    const int b = threadIdx.x;  // bins <= threads
    int here = 0;
    if (b < bins) total[b] = here = prefix_over_warps<kClusterWarps>(count, bins, b);
    cluster_arrive();
    const int staged_at = block_exclusive_scan(here, kClusterWarps, warp_total[0]);
    if (b < bins) local[b] = staged_at;
    cluster_wait();
    int all = 0, before = 0;
    if (b < bins) {
#pragma unroll
      for (int r = 0; r < kEmbedCluster; ++r) {
        const int c = r < blocks ? cluster.map_shared_rank(total, r)[b] : 0;
        all += c;
        before += r < me ? c : 0;
      }
    }
    const int start = block_exclusive_scan(all, kClusterWarps, warp_total[1]);  // its barriers publish local
    if (b < bins) base[b] = start + before - staged_at;
#pragma unroll
    for (int i = 0; i < KPT; ++i) {
      if (key[i] == kNoKey) continue;
      const uint32_t digit = (key[i] >> shift) & (bins - 1);
      staged[local[digit] + count[warp * bins + digit] + rank[i]] = make_uint2(key[i], tok[i]);
    }
    __syncthreads();
    uint2* out = pass & 1 ? p.pairs[1] : p.pairs[0];
    for (int i = threadIdx.x; i < mine; i += kClusterThreads) {
      const uint2 x = staged[i];
      const int at = base[(x.x >> shift) & (bins - 1)] + i;
      if (in_bounds(at, p.N, p.status)) out[at] = x;
      // in the last pass the staged pairs are in the order of their whole keys
      if (pass + 1 == plan.passes && (i == 0 || staged[i - 1].x != x.x)) set_present(p, x.x);
    }
    cluster_arrive();  // the pairs are out, and nobody reads this block's counts any more
    cluster_wait();
  }
}

// More tokens: counts per tile, then for each pass a scan of all tiles' counts and the move of
// the tiles' pairs.
constexpr int kSortThreads = 512, kSortWarps = kSortThreads / 32;

// Counts of the first digit per tile; clears the later digits' counts of this tile.
template <typename I>
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(EmbedParams p, EmbedPlan plan) {
  __shared__ int count[kMaxBins];
  const int bins = 1 << plan.digit;
  launch_dependents();
  clear_present(p, blockIdx.x, gridDim.x);
  for (int i = threadIdx.x; i < bins; i += kSortThreads) count[i] = 0;
  __syncthreads();
  const long long first = (long long)blockIdx.x * plan.tile;
  const long long last = first + plan.tile < p.N ? first + plan.tile : p.N;
  for (long long n = first + threadIdx.x; n < last; n += kSortThreads)
    atomicAdd(&count[token_key<I>(p, n) & (bins - 1)], 1);
  __syncthreads();
  for (int i = threadIdx.x; i < bins; i += kSortThreads) {
    p.hist[(size_t)blockIdx.x * bins + i] = count[i];
    for (int q = 1; q < plan.passes; ++q) p.hist[((size_t)q * plan.tiles + blockIdx.x) * bins + i] = 0;
  }
}

// hist[tile][bin] of one pass becomes the number of the bin's pairs in earlier tiles, totals[bin]
// that in all tiles.  A block takes 32 bins (one per lane), a warp of it four of the tiles.
constexpr int kScanThreads = 1024, kTilesPerWarp = 4;  // 128 tiles at most

__global__ void __launch_bounds__(kScanThreads) sort_scan_kernel(EmbedParams p, EmbedPlan plan, int pass) {
  __shared__ int sum[32][33];
  const int bins = 1 << plan.digit, warp = threadIdx.x / 32, lane = threadIdx.x % 32, b = blockIdx.x * 32 + lane;
  int* hist = p.hist + (size_t)pass * plan.tiles * bins;
  int c[kTilesPerWarp], s = 0;
  launch_dependents();
  wait_for_previous();
#pragma unroll
  for (int i = 0; i < kTilesPerWarp; ++i) {
    const int t = warp * kTilesPerWarp + i;
    c[i] = t < plan.tiles && b < bins ? hist[(size_t)t * bins + b] : 0;
    s += c[i];
  }
  sum[warp][lane] = s;
  __syncthreads();
  int at = 0, all = 0;
#pragma unroll
  for (int w = 0; w < 32; ++w) {
    const int x = sum[w][lane];
    at += w < warp ? x : 0;
    all += x;
  }
  if (b >= bins) return;
#pragma unroll
  for (int i = 0; i < kTilesPerWarp; ++i) {
    const int t = warp * kTilesPerWarp + i;
    if (t < plan.tiles) hist[(size_t)t * bins + b] = at;
    at += c[i];
  }
  if (warp == 0) p.totals[pass * bins + b] = all;
}

// A tile's pairs move to their places for digit `pass`, in rounds of 512 * KPT; the next
// digit's counts are gathered on the way (integers, so their order does not matter).
template <typename I, int KPT>
__global__ void __launch_bounds__(kSortThreads) sort_pass_kernel(EmbedParams p, EmbedPlan plan, int pass) {
  __shared__ unsigned short count[kSortWarps * kMaxBins];
  __shared__ int base[kMaxBins], step[kMaxBins];
  const int bins = 1 << plan.digit, shift = pass * plan.digit;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int* hist = p.hist + ((size_t)pass * plan.tiles + blockIdx.x) * bins;
  int* next = pass + 1 < plan.passes ? p.hist + (size_t)(pass + 1) * plan.tiles * bins : nullptr;
  const uint2* in = pass & 1 ? p.pairs[0] : p.pairs[1];
  uint2* out = pass & 1 ? p.pairs[1] : p.pairs[0];
  __shared__ int warp_total[kSortWarps];
  launch_dependents();
  wait_for_previous();
  {  // a thread takes two consecutive bins
    static_assert(kMaxBins == 2 * kSortThreads, "two bins per thread");
    const int b = 2 * threadIdx.x;
    const int t0 = b < bins ? p.totals[pass * bins + b] : 0, t1 = b + 1 < bins ? p.totals[pass * bins + b + 1] : 0;
    const int start = block_exclusive_scan(t0 + t1, kSortWarps, warp_total);
    if (b < bins) base[b] = start + hist[b];
    if (b + 1 < bins) base[b + 1] = start + t0 + hist[b + 1];
    for (int i = threadIdx.x; i < bins; i += kSortThreads) step[i] = 0;
    __syncthreads();
  }
  const long long first = (long long)blockIdx.x * plan.tile;
  const long long last = first + plan.tile < p.N ? first + plan.tile : p.N;
  for (long long sub = first; sub < last; sub += kSortThreads * KPT) {
    for (int b = threadIdx.x; b < bins; b += kSortThreads) base[b] += step[b];  // each bin by its own thread
    for (int i = threadIdx.x; i < kSortWarps * bins; i += kSortThreads) count[i] = 0;
    uint32_t key[KPT], tok[KPT];
    int rank[KPT];
#pragma unroll
    for (int i = 0; i < KPT; ++i) {
      const long long n = sub + (long long)warp * 32 * KPT + 32 * i + lane;
      key[i] = kNoKey;
      tok[i] = (uint32_t)n;
      if (n < last) {
        if (pass) {
          const uint2 x = in[n];
          key[i] = x.x;
          tok[i] = x.y;
        } else {
          key[i] = token_key<I>(p, n);
        }
      }
    }
    __syncthreads();
    rank_in_warp<KPT>(key, shift, plan.digit, lane, count + warp * bins, rank);
    __syncthreads();
    for (int b = threadIdx.x; b < bins; b += kSortThreads) step[b] = prefix_over_warps<kSortWarps>(count, bins, b);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < KPT; ++i) {
      if (key[i] == kNoKey) continue;
      const uint32_t digit = (key[i] >> shift) & (bins - 1);
      const int at = base[digit] + count[warp * bins + digit] + rank[i];
      if (!in_bounds(at, p.N, p.status)) continue;
      out[at] = make_uint2(key[i], tok[i]);
      if (next) atomicAdd(next + (size_t)(at / plan.tile) * bins + ((key[i] >> (shift + plan.digit)) & (bins - 1)), 1);
    }
    __syncthreads();
  }
}

// The rows' bits, from the sorted pairs of the tiles.
__device__ __forceinline__ const uint2* sorted_pairs(const EmbedParams& p, const EmbedPlan& plan);
__global__ void __launch_bounds__(kSortThreads) mark_present_kernel(EmbedParams p, EmbedPlan plan) {
  launch_dependents();
  wait_for_previous();
  const uint2* pairs = sorted_pairs(p, plan);
  const long long i = (long long)blockIdx.x * kSortThreads + threadIdx.x;
  if (i < p.N && (i == 0 || pairs[i - 1].x != pairs[i].x)) set_present(p, pairs[i].x);
}

// the last pass's output (no index into the parameters, which would copy them to local memory)
__device__ __forceinline__ const uint2* sorted_pairs(const EmbedParams& p, const EmbedPlan& plan) {
  return plan.passes & 1 ? p.pairs[0] : p.pairs[1];
}

// ------------------------------------------------------------------------------------ the sums
// Eight columns per thread: consecutive ones where D is a multiple of 8, else one of every
// tpr.  blockIdx.y is the tile of 8 tpr columns.
constexpr int kSumThreads = 256;
constexpr int kZeroRows = 64;  // table rows per zeroing block, about
constexpr int kJoinThreads = 512;
constexpr int kLongChunks = 8;     // chunks whose long runs one block of the join takes
constexpr int kFold = 64;          // partial sums that are folded into one where a run holds them all
// Chunks from which that is worth a launch (rows of 32).  Ids over a large table, with the fold and
// without: 12288 chunks 82 and 76 us, 20480 chunks 92 and 91, 32768 chunks 107 and 113; over 3000 rows 53
// and 53, 64 and 75, 74 and 97.  Two rows take all: 8192 chunks 33 and 83, 16384 chunks 37 and 145.
constexpr int kFoldFrom = 16384;
constexpr int kShortRun = 8;       // partial sums behind a run's first up to which one thread group joins it

// Eight columns as they lie in memory.
template <typename T>
struct Raw {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void add_to(float (&x)[8]) const {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(v);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x[i] += sizeof(T) == 4 ? __uint_as_float(w[i * sizeof(T) / 4])
                             : __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  }
};

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
  // The finished sum of table row v, which is finished once: nobody else reads or writes the row.
  // (Adding by the memory's own add, which nobody waits for, is 4% faster but treats what the row
  // holds below 2^-126 as zero.)
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

// The table rows without a token become zero.  A warp takes a unit of up to 32 rows and 4 KB at a
// time (380 tokens, 966924 x 11: 33 us; with a row at a time 83.  200000 tokens, 1000000 x 64: 96
// and 125), and consecutive warps consecutive units, so that what is being written at a time
// lies together (blocks with 64 rows each, 192 KB apart, wrote at 3.5 TB/s).
__device__ __forceinline__ void zero_absent_rows(const EmbedParams& p, FastDiv D, int block, int blocks) {
  const int lane = threadIdx.x % 32, warps = blockDim.x / 32;
  if ((int)threadIdx.x >= warps * 32) return;
  // a power of two, so that a unit's bits are in one word; not below 4 where that aligns a unit
  int rows = 32;
  while (rows > (p.D % 4 ? 4 : 1) && rows * p.D > 1024) rows /= 2;
  const uint32_t all = ~0u >> (32 - rows);
  const bool vec_rows = p.D % 4 == 0;
  const long long units = ((long long)p.V + rows - 1) / rows, step = (long long)blocks * warps;
  constexpr int kUnits = 8;  // whose bits are read before the first is written
  for (long long u0 = (long long)block * warps + threadIdx.x / 32; u0 < units; u0 += step * kUnits) {
    uint32_t bits[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const long long r = (u0 + i * step) * rows;
      bits[i] = r < p.V ? p.present[r / 32] >> (r % 32) & all : all;
    }
#pragma unroll 1
    for (int i = 0; i < kUnits; ++i) {
      if (bits[i] == all) continue;
      const long long r = (u0 + i * step) * rows;
      const int n = (int)(p.V - r < rows ? p.V - r : rows) * p.D;  // elements
      float* at = p.d_table + (size_t)r * p.D;
      if (bits[i] == 0) {
        for (int c = lane; c < n / 4; c += 32) reinterpret_cast<float4*>(at)[c] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (lane < n % 4) at[n - 1 - lane] = 0.f;
      } else if (vec_rows) {
        for (int c = lane; c < n / 4; c += 32)
          if (!(bits[i] >> D.div32(4 * c) & 1)) reinterpret_cast<float4*>(at)[c] = make_float4(0.f, 0.f, 0.f, 0.f);
      } else {
        for (int c = lane; c < n; c += 32)
          if (!(bits[i] >> D.div32(c) & 1)) at[c] = 0.f;
      }
    }
  }
}

// Blocks below `zero_blocks` look after the rows without a token; a thread group of the others
// walks the runs of one chunk, eight columns per thread (blockIdx.y: tile of 8 tpr columns).
template <typename T, bool VEC>
__global__ void __launch_bounds__(kSumThreads, 3) embed_sum_kernel(EmbedParams p, EmbedPlan plan, int tpr, int groups,
                                                                   int zero_blocks, FastDiv width) {
  extern __shared__ uint2 staged_pairs[];  // of the block's positions
  const uint2* pairs = sorted_pairs(p, plan);
  launch_dependents();
  wait_for_previous();
  if ((int)blockIdx.x < zero_blocks) {
    if (blockIdx.y == 0) zero_absent_rows(p, width, blockIdx.x, zero_blocks);
    return;
  }
  const long long block = blockIdx.x - zero_blocks;
  const int span = groups * plan.chunk;
  const long long at0 = block * span;
  const uint32_t none = (uint32_t)p.V;  // padding, and what lies behind the last token: sorts behind every id
  for (int i = threadIdx.x; i < span; i += blockDim.x)
    staged_pairs[i] = at0 + i < p.N ? pairs[at0 + i] : make_uint2(none, 0);
  const int group = threadIdx.x / tpr;
  const long long c = block * groups + group, s0 = c * plan.chunk, e0 = s0 + plan.chunk;
  const uint32_t prior = s0 > 0 && s0 < p.N ? pairs[s0 - 1].x : none, after = e0 < p.N ? pairs[e0].x : none;
  __syncthreads();
  if (group >= groups) return;
  const uint2* pair = staged_pairs + group * plan.chunk;
  uint32_t cur = pair[0].x;
  if (cur == none) return;
  const Columns<VEC> col(threadIdx.x - group * tpr, tpr, blockIdx.y, p.D);
  const T* d_out = static_cast<const T*>(p.d_out);
  float* head = p.part + (size_t)c * 2 * p.D;
  bool from_before = prior == cur;
  float acc[8];
  zero8(acc);
  constexpr int kAhead = VEC ? 16 / sizeof(T) : 2;  // rows in flight per thread: 128 bytes of them
  for (int i = 0; i < plan.chunk; i += kAhead) {    // plan.chunk is a multiple of kAhead
    Raw<T> raw[VEC ? kAhead : 1];
    float x[VEC ? 1 : kAhead][8];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const uint2 k = pair[i + j];
      const T* row = d_out + (size_t)k.y * p.D;
      if (VEC) {
        if (k.x != none && col.first < p.D) raw[VEC ? j : 0].load(row + col.first);
      } else if (k.x != none) {
        col.load(row, x[VEC ? 0 : j]);
      }
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const uint32_t k = pair[i + j].x;
      if (k != cur) {
        if (from_before) col.store(head, acc);
        else col.finish(p, cur, acc);
        from_before = false;
        cur = k;
        if (cur == none) return;
        zero8(acc);
      }
      if (VEC) {
        raw[VEC ? j : 0].add_to(acc);
      } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) acc[q] += x[VEC ? 0 : j][q];
      }
    }
  }
  if (from_before) col.store(head, acc);
  else if (after == cur) col.store(head + p.D, acc);  // this chunk's tail
  else col.finish(p, cur, acc);
}

// The runs that cross a chunk's border: the chunk where a run begins holds its first partial
// sum (its tail), the chunks it reaches hold the others (their heads).
struct Runs {
  const uint2* pairs;
  uint32_t none;
  int chunk, chunks;
  // key at the first position of chunk n (`none` behind the last)
  __device__ __forceinline__ uint32_t at(long long n) const { return n < chunks ? pairs[n * chunk].x : none; }
  // the id of the run that begins in chunk c and goes on behind it, or `none`; `far`: the key at
  // the first position of chunk c + 1 + kShortRun.  The loads do not wait for one another.
  __device__ __forceinline__ uint32_t begins(long long c, uint32_t* far) const {
    const bool in = c + 1 < chunks;
    const uint32_t next = at(c + 1), last = in ? pairs[(c + 1) * chunk - 1].x : none;
    const uint32_t prior = in && c ? pairs[c * chunk - 1].x : none;
    *far = at(c + 1 + kShortRun);
    return in && next == last && prior != last ? last : none;
  }
};

// A run of up to kShortRun further partial sums that begins in chunk c: one thread group adds
// them from left to right.
template <bool VEC>
__device__ __forceinline__ void join_short_run(const EmbedParams& p, const Runs& runs, const Columns<VEC>& col, long long c) {
  float acc[8], x[8];
  uint32_t far, key[kShortRun];
#pragma unroll
  for (int n = 0; n < kShortRun; ++n) key[n] = runs.at(c + 1 + n);
  const uint32_t id = runs.begins(c, &far);
  if (id == runs.none || far == id) return;
  int heads = 0;
#pragma unroll
  for (int n = 0; n < kShortRun; ++n) heads += key[n] == id;
  col.load(p.part + ((size_t)c * 2 + 1) * p.D, acc);
#pragma unroll 4
  for (int n = 1; n <= heads; ++n) {
    col.load(p.part + (size_t)(c + n) * 2 * p.D, x);
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[q] += x[q];
  }
  col.finish(p, id, acc);
}

// A group of `width` threads (up to a warp's) holds 8 width columns; blockIdx.y is their tile.
// Blocks below `short_blocks`: one group per chunk adds a run of up to kShortRun further partial
// sums from left to right.  Further blocks look after kLongChunks chunks each and take the
// longer runs that begin there: the block's groups add equal slices of the partial sums, whose
// sums are then added from left to right.
template <bool VEC>
__global__ void __launch_bounds__(kJoinThreads) embed_join_kernel(EmbedParams p, EmbedPlan plan, int width,
                                                                 int short_blocks) {
  __shared__ uint32_t found, ids[kLongChunks];
  __shared__ __align__(16) float slice[kJoinThreads * 8];  // written in 16-byte pieces
  const Runs runs{sorted_pairs(p, plan), (uint32_t)p.V, plan.chunk, plan.chunks};
  const int groups = kJoinThreads / width, group = threadIdx.x / width, gt = threadIdx.x - group * width;
  const Columns<VEC> col(gt, width, blockIdx.y, p.D);
  float acc[8], x[8];
  wait_for_previous();
  if ((int)blockIdx.x < short_blocks) {
    if (group < groups) join_short_run<VEC>(p, runs, col, (long long)blockIdx.x * groups + group);
    return;
  }
  const int slices = groups < 32 ? groups : 32;
  const long long c0 = (long long)(blockIdx.x - short_blocks) * kLongChunks;
  if (threadIdx.x < 32) {
    uint32_t far = runs.none;
    const uint32_t own = threadIdx.x < kLongChunks ? runs.begins(c0 + threadIdx.x, &far) : runs.none;
    const uint32_t some = __ballot_sync(0xffffffffu, own != runs.none && far == own);
    if (threadIdx.x == 0) found = some;
    if (threadIdx.x < kLongChunks) ids[threadIdx.x] = own;
  }
  __syncthreads();
  for (uint32_t left = found; left; left &= left - 1) {
    const long long c = c0 + __ffs(left) - 1;
    const uint32_t id = ids[__ffs(left) - 1];
    long long heads = 0;  // chunks behind c that the run reaches: a prefix, since the keys are sorted
    for (;;) {
      const int got = __syncthreads_count(runs.at(c + 1 + heads + threadIdx.x) == id);
      heads += got;
      if (got < kJoinThreads) break;
    }
    zero8(acc);
    if (group < slices) {
      const long long lo = heads * group / slices, hi = heads * (group + 1) / slices;
      if (group == 0) col.load(p.part + ((size_t)c * 2 + 1) * p.D, acc);
#pragma unroll 8
      for (long long n = lo; n < hi; ++n) {
        col.load(p.part + (size_t)(c + 1 + n) * 2 * p.D, x);
#pragma unroll
        for (int q = 0; q < 8; ++q) acc[q] += x[q];
      }
    }
    store8(slice + 8 * threadIdx.x, acc);
    __syncthreads();
    if (group == 0) {
      for (int g = 1; g < slices; ++g) {
#pragma unroll
        for (int q = 0; q < 8; ++q) acc[q] += slice[8 * (g * width + gt) + q];
      }
      col.finish(p, id, acc);
    }
    __syncthreads();
  }
}

// Adds rows at(lo) .. at(hi - 1) of the partial sums, dealt out to `slices` groups of the block in
// equal runs, from left to right; the sum is group 0's.
template <bool VEC, typename At>
__device__ __forceinline__ void block_sum(const EmbedParams& p, const Columns<VEC>& col, int width, int slices, int n,
                                          At at, float (*slice)[9], float (&acc)[8]) {
  const int group = threadIdx.x / width, gt = threadIdx.x - group * width;
  float x[8];
  zero8(acc);
  if (group < slices) {
    const int lo = (int)((long long)n * group / slices), hi = (int)((long long)n * (group + 1) / slices);
#pragma unroll 8
    for (int i = lo; i < hi; ++i) {
      col.load(p.part + (size_t)at(i) * p.D, x);
#pragma unroll
      for (int q = 0; q < 8; ++q) acc[q] += x[q];
    }
  }
#pragma unroll
  for (int q = 0; q < 8; ++q) slice[threadIdx.x][q] = acc[q];
  __syncthreads();
  if (group == 0) {
    for (int g = 1; g < slices; ++g) {
#pragma unroll
      for (int q = 0; q < 8; ++q) acc[q] += slice[g * width + gt][q];
    }
  }
  __syncthreads();
}

// Where there are many chunks: the heads of chunks 64 k .. 64 k + 63 become one (in the place of
// the first) where they all belong to one run, so that no block of the join adds thousands.
template <bool VEC>
__global__ void __launch_bounds__(kJoinThreads) embed_fold_kernel(EmbedParams p, EmbedPlan plan, int width) {
  __shared__ float slice[kJoinThreads][9];  // the ninth only spreads the banks
  const Runs runs{sorted_pairs(p, plan), (uint32_t)p.V, plan.chunk, plan.chunks};
  launch_dependents();
  wait_for_previous();
  const long long c = (long long)blockIdx.x * kFold;
  const uint32_t id = runs.at(c + kFold - 1);
  if (c == 0 || id == runs.none || runs.at(c) != id || runs.pairs[c * plan.chunk - 1].x != id) return;
  const int groups = kJoinThreads / width;
  const Columns<VEC> col(threadIdx.x % width, width, blockIdx.y, p.D);
  float acc[8];
  block_sum<VEC>(p, col, width, groups < 16 ? groups : 16, kFold, [&](int i) { return (c + i) * 2; }, slice, acc);
  if (threadIdx.x < width) col.store(p.part + (size_t)c * 2 * p.D, acc);
}

// The join of many chunks: further blocks look after `per` chunks each, and the heads have been
// folded.  (With few chunks it takes 15 us where embed_join_kernel takes 11; of 31250 chunks in
// two runs that one took 275 us.)
template <bool VEC>
__global__ void __launch_bounds__(kJoinThreads, 3) embed_join_many_kernel(EmbedParams p, EmbedPlan plan, int width,
                                                                  int short_blocks, int per) {
  __shared__ uint32_t found[kJoinThreads / 32], ids[kJoinThreads];
  __shared__ float slice[kJoinThreads][9];
  const Runs runs{sorted_pairs(p, plan), (uint32_t)p.V, plan.chunk, plan.chunks};
  const int groups = kJoinThreads / width, group = threadIdx.x / width, gt = threadIdx.x - group * width;
  const Columns<VEC> col(gt, width, blockIdx.y, p.D);
  float acc[8];
  wait_for_previous();
  if ((int)blockIdx.x < short_blocks) {
    if (group < groups) join_short_run<VEC>(p, runs, col, (long long)blockIdx.x * groups + group);
    return;
  }
  const long long c0 = (long long)(blockIdx.x - short_blocks) * per;
  {
    uint32_t far = runs.none;
    const bool mine = (int)threadIdx.x < per;
    const uint32_t own = mine ? runs.begins(c0 + threadIdx.x, &far) : runs.none;
    const uint32_t some = __ballot_sync(0xffffffffu, own != runs.none && far == own);
    if (threadIdx.x % 32 == 0) found[threadIdx.x / 32] = some;
    ids[threadIdx.x] = own;
  }
  __syncthreads();
  for (int f = 0; f < kJoinThreads / 32; ++f) {
    for (uint32_t left = found[f]; left; left &= left - 1) {
      const int k = 32 * f + __ffs(left) - 1;
      const long long c = c0 + k;
      const uint32_t id = ids[k];
      // the chunks behind c that the run reaches are [c + 1, end): all threads probe, the next ones
      // first, then the rest at equal distances
      int lo = (int)c + 1, hi = plan.chunks, step = 1;
      while (lo < hi) {
        const int at = lo + ((int)threadIdx.x + 1) * step - 1;
        const int n = __syncthreads_count(at < hi && runs.at(at) == id);  // the keys are sorted: the first n probes
        const long long top = lo + (long long)(n + 1) * step - 1;
        lo += n * step;
        if (n < kJoinThreads && top < hi) hi = (int)top;
        step = (hi - lo + kJoinThreads) / (kJoinThreads + 1);  // at least 1 while lo < hi
      }
      // the tail of c, then the heads: one by one, or by folded groups where the run holds them
      const int first = (int)c + 1, end = lo;
      int a = (first + kFold - 1) / kFold * kFold, b = end / kFold * kFold;
      if (a >= b) a = b = end;
      const int n1 = a - first, n2 = n1 + (b - a) / kFold, n = 1 + n2 + (end - b);
      block_sum<VEC>(p, col, width, groups < 64 ? groups : 64, n, [&](int i) {
        return i == 0 ? 2ll * first - 1 : 2ll * (i <= n1 ? first + i - 1 : i <= n2 ? a + (i - 1 - n1) * kFold : b + (i - 1 - n2));
      }, slice, acc);
      if (group == 0) col.finish(p, id, acc);
    }
  }
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
    embed_fwd_kernel<I, W, T, true><<<blocks, kFwdThreads, 0, stream>>>(p, tile, FastDiv(pieces));
  else
    embed_fwd_kernel<I, W, T, false><<<blocks, kFwdThreads, 0, stream>>>(p, tile, FastDiv(pieces));
  return cudaGetLastError();
}

template <typename I>
cudaError_t embed_fwd_ids(const EmbedParams& p, int table_dtype, int dtype, cudaStream_t stream) {
  if (table_dtype == PRISM_BF16) return embed_fwd_types<I, __nv_bfloat16, __nv_bfloat16>(p, stream);
  if (dtype == PRISM_BF16) return embed_fwd_types<I, float, __nv_bfloat16>(p, stream);
  return embed_fwd_types<I, float, float>(p, stream);
}

// The one-launch sort.  *placed: whether the device has room for its cluster at all, which is certain up
// to the portable size; a device that is cut into parts may not place a larger one.
template <typename I, int KPT>
cudaError_t sort_cluster(const EmbedParams& p, const EmbedPlan& plan, cudaStream_t stream, bool* placed) {
  *placed = plan.cluster <= kPortableCluster || !g_portable_clusters.load(std::memory_order_relaxed);
  if (!*placed) return cudaSuccess;
  auto bytes = [](int digit) { return (size_t)kClusterThreads * KPT * 8 + (((size_t)kClusterWarps * 2 + 12) << digit); };
  cudaError_t err = cudaFuncSetAttribute(sort_cluster_kernel<I, KPT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)bytes(kEmbedMaxDigit));
  if (err == cudaSuccess && plan.cluster > kPortableCluster)
    err = cudaFuncSetAttribute(sort_cluster_kernel<I, KPT>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(plan.cluster);
  cfg.blockDim = dim3(kClusterThreads);
  cfg.dynamicSmemBytes = bytes(plan.digit);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = plan.cluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (plan.cluster > kPortableCluster) {
    int clusters = 0;
    err = cudaOccupancyMaxActiveClusters(&clusters, sort_cluster_kernel<I, KPT>, &cfg);
    if (err != cudaSuccess || clusters < 1) {
      cudaGetLastError();
      *placed = false;
      return cudaSuccess;
    }
  }
  return cudaLaunchKernelEx(&cfg, sort_cluster_kernel<I, KPT>, p, plan);
}

template <typename I, int KPT>
cudaError_t sort_tiles(const EmbedParams& p, const EmbedPlan& plan, cudaStream_t stream) {
  sort_count_kernel<I><<<plan.tiles, kSortThreads, 0, stream>>>(p, plan);
  cudaError_t err = cudaGetLastError();
  const int scans = ((1 << plan.digit) + 31) / 32;
  for (int pass = 0; pass < plan.passes && err == cudaSuccess; ++pass) {
    err = launch_chained(sort_scan_kernel, dim3(scans), kScanThreads, 0, stream, p, plan, pass);
    if (err == cudaSuccess)
      err = launch_chained(sort_pass_kernel<I, KPT>, dim3(plan.tiles), kSortThreads, 0, stream, p, plan, pass);
  }
  if (err == cudaSuccess && p.present)
    err = launch_chained(mark_present_kernel, dim3((int)((p.N + kSortThreads - 1) / kSortThreads)), kSortThreads, 0, stream,
                         p, plan);
  return err;
}

template <typename I>
cudaError_t embed_sort(const EmbedParams& p, EmbedPlan plan, cudaStream_t stream) {
  if (plan.cluster) {
    bool placed;
    const cudaError_t err =
        plan.kpt == 1 ? sort_cluster<I, 1>(p, plan, stream, &placed) : sort_cluster<I, 2>(p, plan, stream, &placed);
    if (placed) return err;
    plan.by_tiles();
  }
  return plan.kpt == 2 ? sort_tiles<I, 2>(p, plan, stream)
         : plan.kpt == 4 ? sort_tiles<I, 4>(p, plan, stream) : sort_tiles<I, 8>(p, plan, stream);
}

template <typename T, bool VEC>
cudaError_t embed_sums(const EmbedParams& p, const EmbedPlan& plan, cudaStream_t stream) {
  const int need = (p.D + 7) / 8;  // threads that hold a row
  const int tpr = need < kSumThreads ? need : kSumThreads;
  // a block's pairs stay within 32 KB of shared memory
  const int most = 4096 / plan.chunk, fit = kSumThreads / tpr, groups = fit < most ? fit : most;
  const int tiles = (need + tpr - 1) / tpr, threads = tpr * groups < 64 ? 64 : tpr * groups;
  const int sum_blocks = (plan.chunks + groups - 1) / groups;
  const int zero_blocks = p.accumulate ? 0 : (int)std::min<long long>(8 * kSMs, ((long long)p.V + kZeroRows - 1) / kZeroRows);
  cudaError_t err = launch_chained(embed_sum_kernel<T, VEC>, dim3(sum_blocks + zero_blocks, tiles), threads,
                                   (size_t)groups * plan.chunk * 8, stream, p, plan, tpr, groups, zero_blocks, FastDiv(p.D));
  if (err != cudaSuccess || plan.chunks == 1) return err;
  const int width = need < 32 ? need : 32, joins = kJoinThreads / width, slabs = (need + width - 1) / width;
  const int short_blocks = (plan.chunks + joins - 1) / joins;
  if (plan.chunks > kFoldFrom) {
    err = launch_chained(embed_fold_kernel<VEC>, dim3(plan.chunks / kFold, slabs), kJoinThreads, 0, stream, p, plan, width);
    if (err != cudaSuccess) return err;
    // few chunks per block where there are few, since a block takes its long runs one by one
    const int per = std::min(std::max(plan.chunks / (8 * kSMs), 8), kJoinThreads);
    return launch_chained(embed_join_many_kernel<VEC>, dim3(short_blocks + (plan.chunks + per - 1) / per, slabs),
                          kJoinThreads, 0, stream, p, plan, width, short_blocks, per);
  }
  const int long_blocks = plan.chunks > kShortRun + 1 ? (plan.chunks + kLongChunks - 1) / kLongChunks : 0;
  return launch_chained(embed_join_kernel<VEC>, dim3(short_blocks + long_blocks, slabs), kJoinThreads, 0, stream, p, plan,
                        width, short_blocks);
}

}  // namespace

void set_portable_clusters(bool on) { g_portable_clusters.store(on, std::memory_order_relaxed); }

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
