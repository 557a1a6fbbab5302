// Sizes, pointers and workspace layout of the embedding kernels.
#pragma once

#include "rowops.cuh"

namespace prism {

constexpr int kEmbedMaxDigit = 10;   // bits of one sorting pass
constexpr int kEmbedCluster = 16;    // most blocks of the one-launch sort
constexpr int kPortableCluster = 8;  // most blocks of a cluster that every device places
constexpr int kEmbedFill = 148 * 2048;
constexpr int kEmbedFwdTile = 256;   // most tokens of a lookup block

// Pointers and sizes of one lookup or gradient call (device pointers).
struct EmbedParams {
  const void* ids;
  const void* table;
  const void* d_out;
  const int32_t* lengths;
  void* out;
  float* d_table;
  uint2* pairs[2];    // backward workspace: (id, token) pairs, the passes' outputs in turn
  int* hist;          // [passes, tiles, bins]: a digit's pairs of a tile, then those of earlier tiles
  int* totals;        // [passes, bins]: a digit's pairs
  uint32_t* present;  // dense gradient: one bit per table row, set where a token names it
  float* part;        // [chunks, 2, D]
  long long N;        // B T < 2^31
  FastDiv T;
  int V, D, accumulate;
  float scale;
  int* status;
};

// How the gradient's sort and sums are cut, and where they work.  Sizes alone decide.
struct EmbedPlan {
  int digit, passes;   // bits of a pass; passes
  int cluster, kpt;    // blocks of the one-launch sort (0: by tiles); pairs per thread of a round
  int tile, tiles;     // tokens of a sorting block; blocks
  int tile_kpt;        // kpt of the sort by tiles
  int chunk, chunks;   // sorted positions that one thread group sums; groups
  size_t off_hist, off_totals, off_present, off_part, off_pairs[2], bytes;
  EmbedPlan(long long N, int V, int D) {
    int bits = 1;
    while (bits < 31 && (V >> bits) != 0) ++bits;  // the keys are 0 .. V
    passes = (bits + kEmbedMaxDigit - 1) / kEmbedMaxDigit;
    digit = (bits + passes - 1) / passes;
    cluster = kpt = 0;
    tile = tiles = tile_kpt = 0;
    if (N <= 1024 * 2 * kEmbedCluster) {
      kpt = N <= 1024 * kEmbedCluster ? 1 : 2;
      cluster = 1;
      while (1024ll * kpt * cluster < N) cluster *= 2;
    }
    if (cluster == 0 || cluster > kPortableCluster) {  // the sort by tiles, if only where the cluster has no place
      // at most 128 tiles, each a multiple of what 512 threads sort at a time
      tile_kpt = N <= 128 * 1024 ? 2 : N <= 128 * 2048 ? 4 : 8;
      const int round = 512 * tile_kpt;
      tile = (int)(((N + 127) / 128 + round - 1) / round * round);
      tiles = (int)((N + tile - 1) / tile);
    }
    if (cluster == 0) kpt = tile_kpt;
    // enough groups of D / 8 threads to fill the SMs, but chunks of at least 16 positions: a run
    // that crosses a chunk's border costs a partial sum (a multiple of 8: the rows in flight)
    const long long need = (D + 7) / 8, c = (N * need + kEmbedFill - 1) / kEmbedFill;
    chunk = c < 16 ? 16 : c > 128 ? 128 : (int)(c + 7) / 8 * 8;
    chunks = (int)((N + chunk - 1) / chunk);
    auto al = [](size_t x) { return (x + 255) & ~(size_t)255; };
    bytes = 0;
    for (size_t& off : off_pairs) { off = bytes; bytes += al((size_t)N * 8); }
    off_hist = bytes; bytes += al(((size_t)passes * tiles << digit) * 4);
    off_totals = bytes; bytes += al(((size_t)passes << digit) * 4);
    off_present = bytes; bytes += al(((size_t)V + 31) / 32 * 4);
    off_part = bytes; bytes += al((size_t)chunks * 2 * D * 4);
  }
  void by_tiles() {
    cluster = 0;
    kpt = tile_kpt;
  }
};

}  // namespace prism
