// The line of tiles that the prefix kernel's pairs of CTAs share out, as the kernel and the join see it.
#pragma once

#include "smla_internal.h"

namespace smla {

constexpr int kPrefixRows = 128;                           // rows of a pair
constexpr uint32_t kExpandedPage = 9 * 8192;               // bytes of 64 positions x 576 dims in fp16

struct Segment {
  int rows, first_row, blocks;                             // rows that see it, the first of them, blocks of 128 rows
  size_t page;                                             // its first expanded page
  bool own;
};

__host__ __device__ __forceinline__ int segments_of(const PrefixParams& p) { return p.prefixes + (p.own ? p.requests : 0); }

__device__ __forceinline__ Segment segment_of(const PrefixParams& p, int g) {
  Segment s;
  s.own = g >= p.prefixes;
  const int r = s.own ? g - p.prefixes : g;
  s.rows = s.own ? p.q_per_req * p.H : p.rows;
  s.first_row = r * s.rows;
  s.blocks = s.own ? p.own_blocks : p.row_blocks;
  s.page = 2 * (s.own ? (size_t)p.prefixes * p.tiles_per_prefix + (size_t)r * p.tiles_per_own : (size_t)r * p.tiles_per_prefix);
  return s;
}

__device__ __forceinline__ int clamped_to(int len, int pages) {
  return (int)min((long long)max(len, 0), (long long)pages * kPageSize);
}

// Positions of a segment: the longest of its queries' lengths; `least`: below which every row sees all.
__device__ __forceinline__ int segment_len(const PrefixParams& p, int g, int* least = nullptr) {
  if (g < p.prefixes) {
    const int n = clamped_to(__ldg(p.lens + g), p.pages);
    if (least) *least = n;
    return n;
  }
  int most = 0, low = 0x7fffffff;
  const int b0 = (g - p.prefixes) * p.q_per_req;
#pragma unroll 1
  for (int b = b0; b < b0 + p.q_per_req; ++b) {
    const int n = clamped_to(__ldg(p.own_lens + b), p.own_pages);
    most = max(most, n);
    low = min(low, n);
  }
  if (least) *least = low;
  return most;
}

__device__ __forceinline__ int tiles_of(int len) { return (int)(((long long)len + kDenseTile - 1) / kDenseTile); }

// The line that is shared out: each item (a segment's block of rows) is `start` units, for what a pair spends on going on to
// it, and then its tiles; none where not every pair has a tile.
constexpr int kPairStart = 4;

__device__ __forceinline__ int item_start(long long tiles, int pairs) { return tiles >= pairs ? kPairStart : 0; }

// Pairs that have a run when U units are shared out over `pairs`, and the first unit of the c-th of them.
__device__ __forceinline__ int active_pairs(long long U, int pairs) { return (int)min((long long)pairs, max(U, 1ll)); }
__device__ __forceinline__ long long pair_start(long long U, int active, int c) {
  const unsigned long long x = (unsigned long long)U * c;
  return x >> 32 ? x / active : (uint32_t)x / (uint32_t)active;
}

}  // namespace smla
