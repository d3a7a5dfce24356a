// Attention of many rows over shared prefixes: the part of the shared decode that is bound by the SM, not by HBM.
//
//   s_t = sm_scale q.k_t,  out = sum_t softmax_t(s) v_t,  lse = ln sum_t exp(s_t)
//
// over the positions of a prefix, for the rows of all requests that share it; short positions of the requests' own go along as
// further segments, each seen by its request's rows.
//
// Expand.  The records are written once as fp16, K' = [code scale | rope] 2^-e, e one exponent per 32 positions that puts
// their largest value into [2^13, 2^14): one rounding of 2^-11 of the value (2^-38 of the largest for the smallest).  It makes up
// nearly all of lse's error (unit records: rms 2e-5 behind 1000 and 2000 positions, 8e-6 .. 1.2e-5 behind 9001, 1e-6 without it;
// the worst of 2048 rows 5e-4, where one position has a fifth of the weight), and buys one product per tile instead of one
// per scale block, whose accumulators do not fit beside O.  The expanded
// pages serve all row blocks, so the conversion is not in the loop that feeds the tensor core.  A page is 9 chunks of 64
// dims, 64 rows of 128 bytes each, 128B-swizzled as in shared memory.
//
// Attention.  A pair of CTAs (a cluster of two, cta_group::2) takes 128 rows, 64 each, through the tiles of 128 positions: 64
// rows are what a CTA's tensor memory holds of O (64 x 512 fp32, half of it) beside two score buffers, and what its shared
// memory holds of q (72 KB) beside the ring of operands.  Scores: M = 128 rows, N = 128 positions; each CTA loads the 9
// chunks of its page.  Values: M = 128, N = 256 dims twice; each CTA loads its 4 chunks of both pages: 136 KB per tile,
// where a CTA alone would need 278 KB for its 64 rows.  TMEM lane l holds row l % 64: the scores of page l / 64, and dims
// 128 (l / 64) .. of each half of the dims.
//   Weights are p = 2^(s + e - R) in fp16, R a power-of-two reference per row that puts the first tile's largest at 2^6 and
// moves when a weight would pass 2^15 (the accumulators are then scaled back); l = sum p 2^-e in fp32.  q is exact in fp16
// but for elements below 2^-20 of their row's largest.
//   The tiles of all (segment, block of 128 rows) items, laid end to end with a few units for each item's start, are
// shared out over the pairs in equal runs; an item that crosses runs leaves fp32 partials for the join.
//
// What bounds it: shared memory.  A tile's operands and copies are 392 KB per CTA (q 72, keys 72, weights 48, values 64, copies
// 136), 3060 cycles at 128 bytes each; measured 3080 (the products alone 2180).  Measured, whole calls: 2048 rows x 32768
// positions with 64 own per request 125 us (146 GFLOP), with 16 .. 1024 own 129 us; of them 13 and 16 the expansion, 9 the join.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <atomic>
#include <cstddef>

#include "smla_dense_parts.cuh"
#include "smla_device.cuh"
#include "smla_internal.h"
#include "smla_prefix_parts.cuh"
#include "smla_ptx.cuh"
#include "smla_split_layout.cuh"

namespace smla {
namespace {

constexpr uint32_t kHalfChunk = kKChunk / 2;               // 64 positions (or rows) x 64 dims fp16

// ----------------------------------------------------------------------------- expand

constexpr int kExpandPart = 32;           // positions with one exponent
// The exponent of positions without values, whose scores are 0.  Any would be right, but the rows' references follow the
// largest s + e: a higher one takes bits from the weights of the others, a lower one leaves too little between a zero's
// weight and the least float where those have large values.  This one leaves all bits beside largest values from 2^-57 to
// 2^49.  (With e = 0 prefixes of values of 2^-42 came out as zeros.)
constexpr int kNoValues = -50;
constexpr int kExpandWarps = 8, kExpandTokens = kExpandPart / kExpandWarps;

// The largest |E4M3| among 16 codes (NaNs count as the largest number).
__device__ __forceinline__ float largest_code(const uint4& v) {
  uint32_t m = __vmaxu4(__vmaxu4(v.x & 0x7f7f7f7fu, v.y & 0x7f7f7f7fu), __vmaxu4(v.z & 0x7f7f7f7fu, v.w & 0x7f7f7f7fu));
  m = __vminu4(m, 0x7e7e7e7eu);
  m = max(max(m & 0xffu, m >> 8 & 0xffu), max(m >> 16 & 0xffu, m >> 24));
  return f16x2_to_f32x2(e4m3x2_to_f16x2((uint16_t)m)).x;
}

// Half a page at a time, 4 positions per warp, 16 latent dims and 2 rope dims per lane.  (32768 positions, with the
// launch: a page per CTA 12.8 us, half a page 13.7, with a lane's 32 bytes stored at once instead of in halves of two sectors
// 10.7: 59 MB, 5.5 TB/s.)  Positions that are no numbers are written as zeros
// and marked, because a weight of 0 would make a NaN of them for the rows that do not see them.
__device__ __forceinline__ void expand_part(const PrefixParams& p, int g, bool own, int part, int len, const int32_t* table,
                                            float* top_s, uint32_t* marks_s, int warp, int lane) {
  const int t0 = part * kExpandPart, lp = part >> 1;
  const bool used = lp * kPageSize < len;
  const int page = used ? __ldg(table + lp) : -1;
  const bool good = page >= 0 && (int64_t)page < p.num_pages;
  if (!good && used && threadIdx.x == 0) atomicOr(p.err, SMLA_DEVERR_PAGE_RANGE);
  uint4 code[kExpandTokens];
  float scale[kExpandTokens];
  uint32_t rope[kExpandTokens];
  const int first = (part & 1) * kExpandPart + warp * kExpandTokens;    // this warp's positions in the page
#pragma unroll
  for (int i = 0; i < kExpandTokens; ++i) {
    code[i] = make_uint4(0u, 0u, 0u, 0u);
    scale[i] = 0.f;
    rope[i] = 0;
    if (!good || t0 + warp * kExpandTokens + i >= len) continue;
    const uint8_t* rec = p.kv + ((int64_t)page * kPageSize + first + i) * kRecordBytes;
    code[i] = ptx::ldg_stream(rec + 16 * lane);
    scale[i] = __ldg(reinterpret_cast<const float*>(rec + kDLatent) + (lane >> 3));
    rope[i] = __ldg(reinterpret_cast<const uint32_t*>(rec + kDLatent + 16) + lane);
  }
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < kExpandTokens; ++i) {
    const float a = largest_code(code[i]) * fabsf(scale[i]), b = fabsf(__uint_as_float(rope[i] << 16)),
                c = fabsf(__uint_as_float(rope[i] & 0xffff0000u));
    const float m = fmaxf(a, fmaxf(b, c));
    if (m < CUDART_INF_F) top = fmaxf(top, m);
  }
  top = ptx::warp_max(top);
  if (lane == 0) top_s[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kExpandWarps; ++w) top = fmaxf(top, top_s[w]);
  const int e = top > 0.f ? min(max((int)(__float_as_uint(top) >> 23) - 127 - 13, -100), 100) : kNoValues;
  const float down = exp2_int(-e);
  const size_t at = segment_of(p, g).page + lp;
  unsigned char* to = p.expanded + at * kExpandedPage;
  uint32_t marks = 0;
#pragma unroll
  for (int i = 0; i < kExpandTokens; ++i) {
    const int t = first + i;
    const uint32_t w[4] = {code[i].x, code[i].y, code[i].z, code[i].w};
    uint32_t o[8], most = 0;
    const float by = scale[i] * down;                      // (exact where the products are above fp16's least)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 a = f16x2_to_f32x2(e4m3x2_to_f16x2((uint16_t)(w[j >> 1] >> (16 * (j & 1)))));
      const float2 b = ptx::unpack2(ptx::mul2(ptx::pack2(a.x, a.y), ptx::pack2(by, by)));
      const __half2 x = __floats2half2_rn(b.x, b.y);
      o[j] = *reinterpret_cast<const uint32_t*>(&x);
      most = __vmaxu2(most, o[j] & 0x7fff7fffu);
    }
    const __half2 rv = __floats2half2_rn(__uint_as_float(rope[i] << 16) * down, __uint_as_float(rope[i] & 0xffff0000u) * down);
    uint32_t ro = *reinterpret_cast<const uint32_t*>(&rv);
    most = __vmaxu2(most, ro & 0x7fff7fffu);
    if (__any_sync(0xffffffffu, __vcmpgeu2(most, 0x7c007c00u) != 0)) {
      marks |= 1u << i;
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = 0;
      ro = 0;
    }
    // the lane's two 16-byte units are one 32-byte sector, swapped in odd rows
    unsigned char* sector = to + (lane >> 2) * kHalfChunk + (swz128(t, (lane & 3) * 2) & ~31u);
    if (t & 1) ptx::stg256(sector, make_uint4(o[4], o[5], o[6], o[7]), make_uint4(o[0], o[1], o[2], o[3]));
    else ptx::stg256(sector, make_uint4(o[0], o[1], o[2], o[3]), make_uint4(o[4], o[5], o[6], o[7]));
    *reinterpret_cast<uint32_t*>(to + kRopeChunk * kHalfChunk + swz128(t, lane >> 2) + (lane & 3) * 4) = ro;
  }
  if (lane == 0) marks_s[warp] = marks;
  __syncthreads();
  if (threadIdx.x < kExpandWarps) {
    marks = __reduce_or_sync((1u << kExpandWarps) - 1u, marks_s[threadIdx.x] << threadIdx.x * kExpandTokens);
    if (threadIdx.x == 0) p.info[2 * at + (part & 1)] = make_int4(e, good, (int)marks, 0);
  }
  __syncthreads();                                         // (the shared values have been read)
}

__global__ void __launch_bounds__(32 * kExpandWarps) expand_kernel(const PrefixParams p, int per_prefix, int per_own) {
  __shared__ float top_s[kExpandWarps];
  __shared__ uint32_t marks_s[kExpandWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) ptx::griddep_launch_dependents();
  // CTAs: per_prefix for each prefix, then per_own for each request
  const bool own = (int)blockIdx.x >= p.prefixes * per_prefix;
  const int x = own ? blockIdx.x - p.prefixes * per_prefix : blockIdx.x, per = own ? per_own : per_prefix;
  const int r = x / per, g = own ? p.prefixes + r : r;
  const int len = segment_len(p, g), pages = own ? p.own_pages : p.pages;
  if (x == r * per && threadIdx.x == 0) {
    bool over = false;
    if (own) {
      for (int b = r * p.q_per_req; b < (r + 1) * p.q_per_req; ++b)
        over |= __ldg(p.own_lens + b) > (long long)p.own_pages * kPageSize;
    } else {
      over = __ldg(p.lens + r) > (long long)p.pages * kPageSize;
    }
    if (over) atomicOr(p.err, SMLA_DEVERR_PAGE_RANGE);
  }
  // (the rest of the last tile is written where no position lies in it, too: zeros, which its weights of 0 meet)
  const int parts = tiles_of(len) * (kDenseTile / kExpandPart);
#pragma unroll 1
  for (int part = x - r * per; part < parts; part += per)
    expand_part(p, g, own, part, len, (own ? p.own_table : p.table) + (size_t)r * pages, top_s, marks_s, warp, lane);
}

// ----------------------------------------------------------------------------- attention

constexpr int kRowsPerCta = kPrefixRows / 2;
constexpr int kSoftWarps = 8;             // warp w: TMEM lanes of quadrant w % 4, half w / 4 of the columns
constexpr int kThreads = 32 * (kSoftWarps + 4);
constexpr int kCopyWarp = kSoftWarps, kQkWarp = kSoftWarps + 1, kPvWarp = kSoftWarps + 2;    // (the second CTA's QK warp
                                                                                             // relays its copies)
constexpr uint64_t kLeastWaitNs = 1000;   // limits below this are meant to run out: nothing is issued

constexpr uint32_t kSlot = 2 * kHalfChunk;                 // ring slot: two of them
constexpr int kRing = 7;
constexpr uint32_t kQ = 0;                                 // 9 half chunks
constexpr uint32_t kP = 9 * kHalfChunk;                    // 2 x [2 position halves][64 rows][64 positions]
constexpr uint32_t kRingAt = kP + 2 * kSlot;
constexpr uint32_t kRope = kRingAt + kRing * kSlot;        // one half chunk
constexpr uint32_t kRed = kRope + kHalfChunk;              // [64 rows][4] float
constexpr uint32_t kSum = kRed + kRowsPerCta * 16;         // [64 rows][4] float
constexpr uint32_t kFactor = kSum + kRowsPerCta * 16;      // [2][64 rows] float
constexpr uint32_t kBar = kFactor + 2 * kRowsPerCta * 4;
constexpr uint32_t kBytes = kBar + 512;
static_assert(kBytes <= 232448, "shared memory");

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kOCol = 0, kSCol = 256;                 // O: two halves of the dims, 128 columns each; scores: 2 x 64

struct Bars {
  uint64_t full[kRing], empty[kRing], rfull, rempty, sfull[2], sempty[2], pfull[2], pfree[2], qfull, drain[2];
  uint32_t tmem;
  int abort;
  int first_segment, first_block, start;   // the item in which the run begins, the units of an item's start
  long long first_begin, run_begin, run_end;   // of its tiles on the line, of the run
  long long sums[kThreads / 32], tiles[kThreads / 32];
};
static_assert(sizeof(Bars) <= 512, "barrier area");

// SMLA_WAIT with the rest of the wait out of line, because code size counts here (2048 rows x 32768 positions, whole call:
// unrolled loops over a tile's slots 245 us, rolled ones 159, and the waits out of line 152), and with tries alone at first.
__device__ __noinline__ uint32_t wait_rest(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
  uint64_t t0 = 0;
  bool ok = false;
#pragma unroll 1
  for (uint32_t n = 1; !ok; ++n) {
    ok = ptx::mbar_try_wait(bar, parity);
    if ((n & 255) == 0 && !ok) {
      const uint64_t now = ptx::globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (*abort || now - t0 > limit_ns) {
        *abort = 1;
        break;
      }
    }
  }
  return __all_sync(0xffffffffu, ok);
}
#undef SMLA_WAIT
#define SMLA_WAIT(bar, par)                                                                               \
  do {                                                                                                    \
    if (__builtin_expect(__any_sync(0xffffffffu, !ptx::mbar_try_wait((bar), (par))), 0)) {                \
      if (ok) ok = wait_rest((bar), (par), &bars->abort, p.wait_ns);                                      \
      asm volatile("" : "+r"(ok));                                                                        \
    }                                                                                                     \
  } while (0)

// Walks the (item, tile) pairs of a run; an item is a segment's block of rows, and may have no tiles.
struct Walk {
  int g, block, t = 0, end = 0, tiles = 0, len = 0;       // tiles t .. end - 1 of the item are in the run
  long long begin;                                         // of the item's tiles on the line
  Segment seg;
  bool entered = false;
  const Bars* bars;
  __device__ __forceinline__ explicit Walk(const Bars* b)
      : g(b->first_segment), block(b->first_block), begin(b->first_begin), bars(b) {}
  __device__ __forceinline__ bool here(const PrefixParams& p) {
    if (__builtin_expect(!entered, 0)) entered = enter(p, begin < bars->run_begin ? (int)(bars->run_begin - begin) : 0);
    return entered;
  }
  // The next item that has tiles; the run's first may have some of them in the run before.
  __device__ __forceinline__ bool enter(const PrefixParams& p, int skip) {
    const int n = segments_of(p), start = bars->start;
    const long long run_end = bars->run_end;
#pragma unroll 1
    for (; g < n; block = 0, ++g) {
      seg = segment_of(p, g);
      len = segment_len(p, g);
      tiles = tiles_of(len);
      if (tiles == 0) continue;
#pragma unroll 1
      for (; block < seg.blocks; ++block, begin += start + tiles, skip = 0) {
        if (begin >= run_end) return false;
        t = skip;
        end = (int)min((long long)tiles, run_end - begin);
        if (t < end) return true;
      }
    }
    return false;
  }
  __device__ __forceinline__ bool last_of_segment() const { return t == end - 1; }
  __device__ __forceinline__ size_t page() const { return seg.page + 2 * (size_t)t; }
  __device__ __forceinline__ void next() {
    if (++t == end) {
      ++block;
      begin += bars->start + tiles;
      entered = false;
    }
  }
};

// One copy of 16 KB per slot: the layout of the expanded pages keeps what a slot takes together.  Returns the slots filled.
__device__ int copy_role(const PrefixParams& p, uint32_t base, Bars* bars, uint32_t rank, int& ropes) {
  Walk w(bars);
  Ring<kRing> k;
  Ring<1> rope;
  uint32_t ok = p.wait_ns >= kLeastWaitNs;
  int filled = 0;
  ptx::griddep_wait();                                     // the expanded pages
  // the values of a tile are loaded behind the keys of the next, in the order of their use
  const unsigned char* before = nullptr;
  auto load = [&](const unsigned char* from) {
    SMLA_WAIT(&bars->empty[k.slot], k.parity ^ 1);
    if (ok && ptx::elect_one()) {
      ptx::mbar_arrive_expect_tx(&bars->full[k.slot], kSlot);
      ptx::bulk_g2s(base + kRingAt + k.slot * kSlot, from, kSlot, &bars->full[k.slot]);
    }
    __syncwarp();
    filled += ok;
    k.next();
  };
  auto values = [&]() {
    const unsigned char* from = before + 2 * rank * kHalfChunk;
#pragma unroll 1
    for (int i = 0; i < 4; ++i) load(from + (i & 1) * kExpandedPage + 4 * (i >> 1) * kHalfChunk);   // dims half i / 2, page i % 2
  };
#pragma unroll 1
  while (w.here(p)) {
    const unsigned char* tile = p.expanded + w.page() * kExpandedPage;
    const bool follows = before != nullptr;
    // a new item's scores wait for its rows, which are loaded after the last one's values were used
    const bool fresh = follows && w.t == 0;
    if (fresh) values();
    const unsigned char* keys = tile + rank * kExpandedPage;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) load(keys + 2 * c * kHalfChunk);
    SMLA_WAIT(&bars->rempty, rope.parity ^ 1);
    if (ok && ptx::elect_one()) {
      ptx::mbar_arrive_expect_tx(&bars->rfull, kHalfChunk);
      ptx::bulk_g2s(base + kRope, keys + kRopeChunk * kHalfChunk, kHalfChunk, &bars->rfull);
    }
    __syncwarp();
    ropes += ok;
    rope.next();
    if (follows && !fresh) values();
    before = tile;
    w.next();
  }
  if (before) values();
  return filled;
}

// The second CTA tells the first, whose warp issues the MMAs, that its operands have landed.
__device__ void relay_role(const PrefixParams& p, uint32_t base, Bars* bars) {
  Walk w(bars);
  Ring<kRing> k;
  Ring<1> rope;
  uint32_t ok = p.wait_ns >= kLeastWaitNs;
  const uint32_t full = ptx::mapa(ptx::smem_u32(&bars->full[0]), 0), rfull = ptx::mapa(ptx::smem_u32(&bars->rfull), 0);
  bool follows = false;
  auto pass = [&](int n) {
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      SMLA_WAIT(&bars->full[k.slot], k.parity);
      if (ok && ptx::elect_one()) ptx::mbar_arrive_cluster(full + 8 * k.slot);
      __syncwarp();
      k.next();
    }
  };
#pragma unroll 1
  while (w.here(p)) {
    const bool fresh = follows && w.t == 0;
    if (fresh) pass(4);
    pass(4);
    SMLA_WAIT(&bars->rfull, rope.parity);
    if (ok && ptx::elect_one()) ptx::mbar_arrive_cluster(rfull);
    __syncwarp();
    rope.next();
    if (follows && !fresh) pass(4);
    follows = true;
    w.next();
  }
  if (follows) pass(4);
}

// Scores and values are issued by a warp each, so that what one waits for hides behind the other's products.  Both follow
// the ring in the order of the copies and pass over each other's slots.
__device__ void qk_role(const PrefixParams& p, uint32_t base, uint32_t tmem, Bars* bars) {
  constexpr uint32_t kIdesc = ptx::idesc_f16(128, 128, 0, 0);
  Walk w(bars);
  Ring<kRing> k;
  Ring<1> rope;
  Ring<2> s;
  uint32_t qpar = 0, ok = p.wait_ns >= kLeastWaitNs;
  bool follows = false;
  const uint64_t dq = ptx::sw128_desc(base + kQ, 16, 1024);
#pragma unroll 1
  while (w.here(p)) {
    const bool fresh = follows && w.t == 0;
    if (fresh) k.skip(4);
    if (!follows || fresh) {                               // an item's rows
      SMLA_WAIT(&bars->qfull, qpar);
      qpar ^= 1;
    }
    SMLA_WAIT(&bars->sempty[s.slot], s.parity ^ 1);
    const uint32_t d = tmem + kSCol + 64 * s.slot;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      SMLA_WAIT(&bars->full[k.slot], k.parity);
      ptx::tc_fence_after();
      const uint32_t ks = k.slot;
      if (ok && ptx::elect_one()) {
        const uint64_t dk = ptx::sw128_desc(base + kRingAt + ks * kSlot, 16, 1024);
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            ptx::mma_f16_ss_pair(d, dq + (uint64_t)((2 * c + x) * (kHalfChunk >> 4) + 2 * kk),
                                 dk + (uint64_t)(x * (kHalfChunk >> 4) + 2 * kk), kIdesc, c + x + kk > 0);
        ptx::mma_commit_pair(&bars->empty[ks]);
      }
      __syncwarp();
      k.next();
    }
    SMLA_WAIT(&bars->rfull, rope.parity);
    ptx::tc_fence_after();
    const uint32_t ss = s.slot;
    if (ok && ptx::elect_one()) {
      const uint64_t dk = ptx::sw128_desc(base + kRope, 16, 1024);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        ptx::mma_f16_ss_pair(d, dq + (uint64_t)(8 * (kHalfChunk >> 4) + 2 * kk), dk + 2 * kk, kIdesc, 1);
      ptx::mma_commit_pair(&bars->rempty);
      ptx::mma_commit_pair(&bars->sfull[ss]);
    }
    __syncwarp();
    rope.next();
    s.next();
    if (follows && !fresh) k.skip(4);
    follows = true;
    w.next();
  }
  if (ptx::elect_one()) ptx::mma_commit_pair(&bars->drain[0]);
  __syncwarp();
}

__device__ void pv_role(const PrefixParams& p, uint32_t base, uint32_t tmem, Bars* bars) {
  constexpr uint32_t kIdesc = ptx::idesc_f16(128, 256, 0, 1);
  Walk w(bars);
  Ring<kRing> k;
  Ring<2> pb;
  uint32_t ok = p.wait_ns >= kLeastWaitNs;
  bool follows = false;
  uint32_t more = 0;                                       // accumulate: not the segment's first tile
  auto values = [&]() {
    SMLA_WAIT(&bars->pfull[pb.slot], pb.parity);
    ptx::tc_fence_after();
    const uint64_t dp = ptx::sw128_desc(base + kP + pb.slot * kSlot, 16, 1024);
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {                          // dims half i / 2, positions half i % 2
      SMLA_WAIT(&bars->full[k.slot], k.parity);
      ptx::tc_fence_after();
      const uint32_t ks = k.slot, ps = pb.slot, acc = more;
      if (ok && ptx::elect_one()) {
        const uint64_t dv = ptx::sw128_desc(base + kRingAt + ks * kSlot, kHalfChunk, 1024);
        const uint32_t d = tmem + kOCol + 128 * (i >> 1);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          ptx::mma_f16_ss_pair(d, dp + (uint64_t)((i & 1) * (kHalfChunk >> 4) + 2 * kk), dv + (uint64_t)(128 * kk), kIdesc,
                               (i & 1) + kk > 0 ? 1 : acc);
        ptx::mma_commit_pair(&bars->empty[ks]);
        if (i == 3) ptx::mma_commit_pair(&bars->pfree[ps]);
      }
      __syncwarp();
      k.next();
    }
    pb.next();
    more = 1;
  };
#pragma unroll 1
  while (w.here(p)) {
    const bool fresh = follows && w.t == 0;
    if (fresh) {
      values();
      more = 0;
    }
    k.skip(4);
    if (follows && !fresh) values();
    follows = true;
    w.next();
  }
  if (follows) values();
  if (ptx::elect_one()) ptx::mma_commit_pair(&bars->drain[1]);
  __syncwarp();
}

// 64 rows of q as fp16 times 2^-x, x per row such that its largest element lies in [2^3, 2^4); the rows' factors
// 2^x sm_scale log2 e to buffer `buf`: the warps of the other 32 rows may not have read the item's before, as nothing but an
// item's start joins the two.  A row with an infinity becomes NaN.  One row at a time, the next two's loads in flight: straight
// code for a warp's eight rows took 11000 cycles instead of 5300, most of them for its instructions.
__device__ __forceinline__ void load_q(const PrefixParams& p, int first, int rows, unsigned char* sm, uint32_t base, int buf,
                                       int warp, int lane) {
  constexpr int kRows = kRowsPerCta / kSoftWarps;
  float* f = reinterpret_cast<float*>(sm + kFactor) + buf * kRowsPerCta;
  const uint4* src = reinterpret_cast<const uint4*>(p.q + (size_t)(first + warp * kRows) * kDQK) + lane;
  const int here = rows - warp * kRows;                    // of this warp's rows
  auto read = [&](int i, uint4 (&to)[3]) {
    const uint4* from = src + (size_t)i * (kDQK / 8);
    to[0] = to[1] = to[2] = make_uint4(0u, 0u, 0u, 0u);
    if (i < min(here, kRows)) {
      to[0] = __ldg(from);
      to[1] = __ldg(from + 32);
      if (lane < 8) to[2] = __ldg(from + 64);
    }
  };
  uint4 n[3], nn[3];
  read(0, n);
  read(1, nn);
#pragma unroll 1
  for (int i = 0; i < kRows; ++i) {
    const uint4 v[3] = {n[0], n[1], n[2]};
#pragma unroll
    for (int j = 0; j < 3; ++j) n[j] = nn[j];
    read(i + 2, nn);
    uint32_t most = 0;                                     // bf16 magnitudes, pairs
#pragma unroll
    for (int j = 0; j < 3; ++j)
      most = __vmaxu2(most, __vmaxu2(__vmaxu2(v[j].x & 0x7fff7fffu, v[j].y & 0x7fff7fffu),
                                     __vmaxu2(v[j].z & 0x7fff7fffu, v[j].w & 0x7fff7fffu)));
    const uint32_t top = __reduce_max_sync(0xffffffffu, max(most & 0xffffu, most >> 16)) << 16;
    const int x = top != 0 ? min(max((int)(top >> 23) - 127 - 3, -120), 120) : 0;
    const float down = top >= 0x7f800000u ? CUDART_NAN_F : exp2_int(-x);
    const int r = warp * kRows + i;
    if (lane == 0) f[r] = exp2_int(x) * (p.sm_scale * kLog2e);
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
      uint32_t o[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const __half2 hv = __floats2half2_rn(__uint_as_float(w[m] << 16) * down, __uint_as_float(w[m] & 0xffff0000u) * down);
        o[m] = *reinterpret_cast<const uint32_t*>(&hv);
      }
      if (j < 2 || lane < 8)
        ptx::sts128(base + kQ + (4 * j + (lane >> 3)) * kHalfChunk + swz128(r, lane & 7), make_uint4(o[0], o[1], o[2], o[3]));
    }
  }
}

__device__ void softmax_role(const PrefixParams& p, unsigned char* sm, uint32_t base, uint32_t tmem, Bars* bars, int warp,
                             int lane, uint32_t rank) {
  const int quad = warp & 3, half = warp >> 2;             // lanes 32 quad .., columns of this half
  const int row = 32 * (quad & 1) + lane, side = quad >> 1;             // of the CTA's 64; positions 64 side .., dims 128 side ..
  const int bar = 1 + (quad & 1);                          // the four warps that share 32 rows
  const uint32_t lane_base = tmem + ((uint32_t)(32 * quad) << 16);
  const uint32_t red = base + kRed + row * 16, sums = base + kSum + row * 16;
  const int part = 2 * side + half;
  const uint32_t to_p = ptx::mapa(ptx::smem_u32(&bars->pfull[0]), 0), to_s = ptx::mapa(ptx::smem_u32(&bars->sempty[0]), 0),
                 to_q = ptx::mapa(ptx::smem_u32(&bars->qfull), 0);
  Walk w(bars);
  Ring<2> s, pb;
  uint32_t ok = p.wait_ns >= kLeastWaitNs;
  int row_len = 0;                                         // positions that this thread's row sees
  float f = 0.f, ref = -CUDART_INF_F, l = 0.f;
  bool first = true, begins = false;
  int buf = 0;                                             // of the item's factors
  Ring<2> last;                                            // the P buffer of the tile before
  int4 next_info = make_int4(0, 0, 0, 0);
  // results of the segment before, written beside the next one's first scores: their place, its rows
  bool pending = false, whole = false;
  size_t to_row = 0;
  int to_rows = 0;
#pragma unroll 1
  for (;;) {
    const bool more = w.here(p);
    const int row0 = w.block * kPrefixRows + rank * kRowsPerCta;        // of the segment's rows
    const int rows = min(kRowsPerCta, w.seg.rows - row0);  // (none, or fewer than none, in a block of at most 64)
    if (more && first) {
      // (every score of the last segment was computed, so no product reads its rows)
      buf ^= 1;
      load_q(p, w.seg.first_row + row0, rows, sm, base, buf, warp, lane);
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (ok && lane == 0) ptx::mbar_arrive_cluster(to_q);
    }
    if (pending) {
      // the segment's results: normalised rows and their lse
      ptx::sts32f(sums + part * 4, l);
      ptx::named_bar_sync(bar, 128);
      const float4 l4 = ptx::lds128f(sums);
      const float z = (l4.x + l4.y) + (l4.z + l4.w);
      const bool none = ref == -CUDART_INF_F && z == 0.f;
      const float lse = none ? -CUDART_INF_F : (ref + log2f(z)) * kLn2, inv = none ? 0.f : 1.f / z;
      if (row < to_rows && part == 0) (whole ? p.lse32 : p.slots_lse)[to_row + row] = lse;
      // 32 rows x 32 dims at a time through the P buffers, which nobody writes before the next item's rows are there:
      // whole lines to global memory (16 bytes of a row per lane: 12800 cycles instead of 7400)
      float* o_to = (whole ? p.out32 : p.slots) + (to_row + row - lane) * kDLatent + 256 * half + 128 * side;
      const uint32_t stage = base + kP + warp * 4096;
      const int most = to_rows - 32 * (quad & 1);          // of these 32 rows
      SMLA_WAIT(&bars->pfree[last.slot], last.parity);
      ptx::tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t o[32];
        ptx::tmem_ld32(lane_base + kOCol + 128 * half + 32 * c, o);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int u = 0; u < 8; ++u)
          ptx::sts128f(stage + swz128(lane, u), __uint_as_float(o[4 * u]) * inv, __uint_as_float(o[4 * u + 1]) * inv,
                       __uint_as_float(o[4 * u + 2]) * inv, __uint_as_float(o[4 * u + 3]) * inv);
        __syncwarp();
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int r = 4 * u + (lane >> 3);
          const float4 x = ptx::lds128f(stage + swz128(r, lane & 7));
          if (r < most) *reinterpret_cast<float4*>(o_to + (size_t)r * kDLatent + 32 * c + 4 * (lane & 7)) = x;
        }
        __syncwarp();
      }
      ptx::tc_fence_before();
      pending = false;
    }
    if (!more) break;
    // this thread's 32 positions, read a tile ahead
    const int4* infos = p.info + 2 * (w.page() + side) + half;
    if (first) {
      ptx::griddep_wait();                                 // (done for a run's later segments)
      next_info = __ldcg(infos);
    }
    const int4 info = next_info;
    if (!w.last_of_segment()) next_info = __ldcg(infos + 4);
    if (first) {
      ptx::named_bar_sync(3, kSoftWarps * 32);             // the rows' factors are written, the results before have left
      f = ptx::lds32f(base + kFactor + (buf * kRowsPerCta + row) * 4);
      row_len = w.len;
      if (w.seg.own && row < rows)
        row_len = clamped_to(__ldg(p.own_lens + (w.g - p.prefixes) * p.q_per_req + (row0 + row) / p.H), p.own_pages);
      begins = w.t == 0;
      ref = -CUDART_INF_F;
      l = 0.f;
    }
    // scores + e in units of log2, 32 positions of this thread's row
    SMLA_WAIT(&bars->sfull[s.slot], s.parity);
    ptx::tc_fence_after();
    uint64_t v[16];
    {
      uint32_t x[32];
      ptx::tmem_ld32(lane_base + kSCol + 64 * s.slot + 32 * half, x);
      ptx::tmem_wait_ld();
      ptx::tc_fence_before();
      __syncwarp();
      if (ok && lane == 0) ptx::mbar_arrive_cluster(to_s + 8 * s.slot);
      s.next();
      const float fe = f * exp2_int(info.x), e = (float)info.x;
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = ptx::fma2(ptx::pack2(x[2 * i], x[2 * i + 1]), ptx::pack2(fe, fe), ptx::pack2(e, e));
    }
    const int left = row_len - w.t * kDenseTile - 64 * side - 32 * half;    // of this thread's 32 positions
    const bool here = info.y;
    if (__builtin_expect(left < 32 || !here, 0)) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float2 d = ptx::unpack2(v[i]);
        if (!here || 2 * i >= left) d.x = -CUDART_INF_F;
        if (!here || 2 * i + 1 >= left) d.y = -CUDART_INF_F;
        v[i] = ptx::pack2(d.x, d.y);
      }
    }
    const uint32_t marks = info.z;
    if (__builtin_expect(marks != 0, 0)) {                 // positions that are no numbers
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float2 d = ptx::unpack2(v[i]);
        if ((marks >> (2 * i) & 1) && 2 * i < left) d.x = CUDART_NAN_F;
        if ((marks >> (2 * i + 1) & 1) && 2 * i + 1 < left) d.y = CUDART_NAN_F;
        v[i] = ptx::pack2(d.x, d.y);
      }
    }
    float top = -CUDART_INF_F;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 d = ptx::unpack2(v[i]);
      top = fmaxf(top, fmaxf(d.x, d.y));
    }
    // R moves when a weight would pass 2^15
    if (ptx::named_bar_or(bar, 128, top > ref + 15.f || (first && top > -CUDART_INF_F))) {
      ptx::sts32f(red + part * 4, top);
      ptx::named_bar_sync(bar, 128);
      const float4 m4 = ptx::lds128f(red);
      const float m = fmaxf(fmaxf(m4.x, m4.y), fmaxf(m4.z, m4.w));
      float by = 1.f;
      if (m > ref + 15.f || (ref == -CUDART_INF_F && m > -CUDART_INF_F)) {
        const float next = ceilf(fminf(m, 3.0e38f)) - 6.f;
        by = ref == -CUDART_INF_F ? 0.f : ptx::ex2_approx(ref - next);         // (a power of two, or 0)
        ref = next;
        l *= by;
      }
      if (!first && __any_sync(0xffffffffu, by != 1.f)) {
        SMLA_WAIT(&bars->pfree[last.slot], last.parity);
        ptx::tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t o[32];
          const uint32_t at = lane_base + kOCol + 128 * half + 32 * c;
          ptx::tmem_ld32(at, o);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * by);
          ptx::tmem_st32(at, o);
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
      }
    }
    {
      const float minus = ref == -CUDART_INF_F ? 0.f : -ref;
      uint64_t sum = 0;
      uint32_t o[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float2 d = ptx::unpack2(ptx::add2(v[i], ptx::pack2(minus, minus)));
        const float a = ptx::ex2_approx(d.x), b = ptx::ex2_approx(d.y);
        sum = ptx::add2(sum, ptx::pack2(a, b));
        const __half2 hv = __floats2half2_rn(a, b);
        o[i] = *reinterpret_cast<const uint32_t*>(&hv);
      }
      const float2 t = ptx::unpack2(sum);
      l = fmaf(t.x + t.y, exp2_int(-info.x), l);
      SMLA_WAIT(&bars->pfree[pb.slot], pb.parity ^ 1);
      const uint32_t dst = base + kP + pb.slot * kSlot + side * kHalfChunk;
#pragma unroll
      for (int u = 0; u < 4; ++u)
        ptx::sts128_async_only(dst + swz128(row, 4 * half + u), make_uint4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]));
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (ok && lane == 0) ptx::mbar_arrive_cluster(to_p + 8 * pb.slot);
      last = pb;
      pb.next();
    }
    first = w.last_of_segment();
    if (first) {
      whole = begins && w.t == w.tiles - 1;
      to_row = whole ? (w.seg.own ? 0 : p.all_rows) + w.seg.first_row + row0
                     : ((size_t)2 * (blockIdx.x >> 1) + (begins ? 1 : 0)) * kPrefixRows + rank * kRowsPerCta;
      to_rows = ok ? rows : 0;
      pending = true;
    }
    w.next();
  }
}

// This pair's run of the line [U c / n, U (c + 1) / n).  The first CTA leaves the segments' places on it for the join.
__device__ __forceinline__ void find_run(const PrefixParams& p, Bars* bars) {
  const int n = segments_of(p), per = (n + kThreads - 1) / kThreads, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g0 = min(n, (int)threadIdx.x * per), g1 = min(n, g0 + per);
  long long tiles = 0, items = 0;
  int last = 0;                                            // tiles of this thread's last segment, mostly its only one
#pragma unroll 1
  for (int g = g0; g < g1; ++g) {
    const int blocks = segment_of(p, g).blocks;
    last = tiles_of(segment_len(p, g));
    tiles += (long long)last * blocks;
    if (last > 0) items += blocks;
  }
  long long all_tiles = tiles;
#pragma unroll
  for (int o = 16; o; o >>= 1) all_tiles += __shfl_xor_sync(0xffffffffu, all_tiles, o);
  if (lane == 0) bars->tiles[warp] = all_tiles;
  if (threadIdx.x == 0) {
    bars->first_segment = n;
    bars->run_begin = bars->run_end = bars->first_begin = bars->first_block = 0;
  }
  __syncthreads();
  all_tiles = 0;
#pragma unroll 1
  for (int x = 0; x < kThreads / 32; ++x) all_tiles += bars->tiles[x];
  const int start = item_start(all_tiles, p.pairs);
  const long long mine = tiles + start * items;
  long long upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += up;
  }
  if (lane == 31) bars->sums[warp] = upto;
  __syncthreads();
  long long total = 0, before = upto - mine;
#pragma unroll 1
  for (int x = 0; x < kThreads / 32; ++x) {
    total += bars->sums[x];
    if (x < warp) before += bars->sums[x];
  }
  const int active = active_pairs(total, p.pairs), c = blockIdx.x >> 1;
  const long long a = c < active ? pair_start(total, active, c) : total, e = c < active ? pair_start(total, active, c + 1) : total;
  const bool starts = a < e && before <= a && a < before + mine;       // the run begins in one of this thread's segments
  if (starts || blockIdx.x == 0) {
#pragma unroll 1
    for (int g = g0; g < g1; ++g) {
      const int x = g == g1 - 1 ? last : tiles_of(segment_len(p, g));
      const long long all = x > 0 ? (long long)(start + x) * segment_of(p, g).blocks : 0;
      if (starts && a >= before && a < before + all) {
        const int block = (int)((a - before) / (start + x));
        bars->first_segment = g;
        bars->first_block = block;
        bars->first_begin = before + (long long)block * (start + x) + start;
        bars->run_begin = a;
        bars->run_end = e;
      }
      if (blockIdx.x == 0) p.begins[g] = before;
      before += all;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
      p.begins[n] = total;
      p.begins[n + 1] = start;
    }
  }
  if (threadIdx.x == 0) bars->start = start;
  __syncthreads();
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) prefix_kernel(const PrefixParams p) {
  extern __shared__ __align__(1024) unsigned char sm[];
  const uint32_t base = ptx::smem_u32(sm);
  Bars* bars = reinterpret_cast<Bars*>(sm + kBar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_ctarank();
  if (threadIdx.x == 0) ptx::griddep_launch_dependents();
  if (warp == kCopyWarp) {
    constexpr int kBars = offsetof(Bars, tmem) / 8;
    // arrivals of the softmax warps of both CTAs, and of the copies of both
    constexpr uint64_t kBySoftmax = (3ull << offsetof(Bars, sempty) / 8) | (3ull << offsetof(Bars, pfull) / 8) |
                                    (1ull << offsetof(Bars, qfull) / 8);
    constexpr uint64_t kByCopies = (((1ull << kRing) - 1) << offsetof(Bars, full) / 8) | (1ull << offsetof(Bars, rfull) / 8);
    static_assert(kBars <= 64, "one bit per barrier");
    for (int i = lane; i < kBars; i += 32)
      ptx::mbar_init(reinterpret_cast<uint64_t*>(bars) + i,
                     kBySoftmax >> i & 1 ? 2 * kSoftWarps : kByCopies >> i & 1 ? (rank == 0 ? 2 : 1) : 1);
    if (lane == 0) bars->abort = p.wait_ns < kLeastWaitNs;
    ptx::fence_mbar_init();
  }
  if (warp == kQkWarp) {
    ptx::tmem_alloc_pair(&bars->tmem, kTmemCols);
    ptx::tmem_relinquish_pair();
  }
  find_run(p, bars);
  ptx::tc_fence_before();
  ptx::cluster_sync_all();                                 // both CTAs' barriers are set up
  ptx::tc_fence_after();
  const uint32_t tmem = bars->tmem;

  int filled = 0, ropes = 0;
  if (warp < kSoftWarps) softmax_role(p, sm, base, tmem, bars, warp, lane, rank);
  else if (warp == kCopyWarp) filled = copy_role(p, base, bars, rank, ropes);
  else if (warp == kQkWarp && rank == 0) qk_role(p, base, tmem, bars);
  else if (warp == kPvWarp && rank == 0) pv_role(p, base, tmem, bars);
  else if (warp == kQkWarp) relay_role(p, base, bars);

  // nothing of the pair's may be in flight when a CTA leaves: the MMAs (their last commit reaches both) and, after a wait
  // that gave up, the copies
  ptx::tc_fence_before();
  __syncthreads();
  int never = 0;
  if (warp == kCopyWarp && bars->abort) {
    // (the first CTA's slots also wait for the second's copies, so the phase of one may stay open: 100 ms then)
    for (int i = max(0, filled - kRing); i < filled; ++i)
      ptx::mbar_wait_warp(&bars->full[i % kRing], (uint32_t)(i / kRing) & 1u, &never, lane, 100000000ull);
    if (ropes > 0) ptx::mbar_wait_warp(&bars->rfull, (uint32_t)(ropes - 1) & 1u, &never, lane, 100000000ull);
  }
  if (warp == kQkWarp) {
    ptx::mbar_wait_warp(&bars->drain[0], 0, &never, lane, 100000000ull);
    ptx::mbar_wait_warp(&bars->drain[1], 0, &never, lane, 100000000ull);
    ptx::tc_fence_after();
  }
  if (threadIdx.x == 0 && bars->abort) atomicOr(p.err, SMLA_DEVERR_TIMEOUT);
  ptx::cluster_sync_all();
  if (warp == kQkWarp) ptx::tmem_dealloc_pair(tmem, kTmemCols);
}

}  // namespace

cudaError_t launch_prefix(const PrefixParams& p, cudaStream_t stream) {
  static std::atomic<bool> set[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !set[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(prefix_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    if (e != cudaSuccess) return e;
    if (dev < 64) set[dev].store(true, std::memory_order_relaxed);
  }
  // a CTA per half page, up to about eight per SM (tables are often far wider than what is in them)
  auto ctas = [&](int segments, int tiles) {
    const long long room = (16ll * p.pairs + segments - 1) / segments, parts = 4ll * tiles;
    return (int)(parts < room ? parts : room);
  };
  const int per_prefix = ctas(p.prefixes, p.tiles_per_prefix), per_own = p.own ? ctas(p.requests, p.tiles_per_own) : 0;
  expand_kernel<<<p.prefixes * per_prefix + (p.own ? p.requests * per_own : 0), 32 * kExpandWarps, 0, stream>>>(p, per_prefix,
                                                                                                              per_own);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * p.pairs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = a;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prefix_kernel, p);
}

}  // namespace smla
