// Sizes, pointers and workspace layout of the embedding kernels.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace prism {

constexpr int kEmbedMaxDigit = 10;   // bits of one sorting pass
constexpr int kEmbedFwdTile = 256;   // most tokens of a lookup block

// Pointers and sizes of one lookup or gradient call (device pointers).
struct EmbedParams {
  const void* ids;
  const void* table;
  const void* d_out;
  const int32_t* lengths;
  void* out;
  float* d_table;
  uint32_t* keys[2];  // backward workspace: ids and token numbers, in turn
  uint32_t* toks[2];
  int* hist;          // [passes, tiles, bins]
  float* part;        // [chunks, 2, D]
  long long N;        // B T < 2^31
  int T, V, D, accumulate;
  float scale;
  int* status;
};

// How the gradient's sort and sums are cut, and where they work.  Sizes alone decide.
struct EmbedPlan {
  int digit, passes;        // bits of a pass; passes
  int tile, tiles, rounds;  // tokens of a sorting block; blocks; pairs per thread and round
  int chunk, chunks;        // sorted positions that one thread group sums; groups
  size_t off_hist, off_part, off_pairs[4], bytes;
  EmbedPlan(long long N, int V, int D) {
    int bits = 1;
    while (bits < 31 && (V >> bits) != 0) ++bits;  // the keys are 0 .. V
    passes = (bits + kEmbedMaxDigit - 1) / kEmbedMaxDigit;
    digit = (bits + passes - 1) / passes;
    // every sorting block reads the counts of all tiles, so there are at most 128 of them
    if (N <= 128 * 1024) {
      rounds = 2;
      tile = 1024;
    } else {
      rounds = 8;
      tile = (int)(((N + 127) / 128 + 4095) / 4096 * 4096);
    }
    tiles = (int)((N + tile - 1) / tile);
    // about 2048 groups, so that every SM has some; runs of more than a chunk cost partial sums
    const long long c = (N + 2047) / 2048;
    chunk = c < 8 ? 8 : c > 128 ? 128 : (int)c;
    chunks = (int)((N + chunk - 1) / chunk);
    auto al = [](size_t x) { return (x + 255) & ~(size_t)255; };
    bytes = 0;
    for (size_t& off : off_pairs) { off = bytes; bytes += al((size_t)N * 4); }
    off_hist = bytes; bytes += al(((size_t)passes * tiles << digit) * 4);
    off_part = bytes; bytes += al((size_t)chunks * 2 * D * 4);
  }
};

}  // namespace prism
