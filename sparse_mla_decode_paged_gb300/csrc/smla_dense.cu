// Dense decode attention over the paged FP8 latent cache: every cached position of a request attends
// (no top-k list).
//
//   s_t = sm_scale q.k_t,  out = sum_t softmax_t(s) v_t,  lse = ln sum_t exp(s_t),
//   k = [e4m3(code_d) scale_{d/128}, d < 512 | rope, 64], v = k[0..511].
//
// A request's rows (its queries' heads) form groups of NR = 16, 32 or 64 rows; an item is one (request, row
// group), a tile 128 positions (two pages) of an item.  The tiles of all items, laid end to end, are shared
// out over the CTAs in runs of equal time (from seq_lens, on the device), so a ragged batch or a single long request
// keeps every SM busy; an item that crosses a CTA boundary leaves partial results that the merge kernel joins.
//
// Scores.  The codes go to the tensor core as they are (kind::f8f6f4), with no conversion: q is split into
// two E4M3 terms, q 2^-x = hi + lo with x chosen per row so that its largest latent element lies in [2^7, 2^8).  hi
// keeps 4 significant bits and lo the other 4 of a bf16 value, so the split is exact but for elements below
// about 2^-9 of the largest (their error is below 2^-17 of it, 2^-8 of that element's own bf16 rounding).  S^T of
// a tile: M = 128 positions, one accumulator per 128-dim scale block; for up to 32 rows hi and lo are one MMA of N = 2 NR
// columns and meet in the softmax threads, for 64, where TMEM is full, two MMAs into NR columns.  The softmax threads
// form s = 2^x sum_b (S_hi + S_lo) scale_b in fp32.  The rope part is a bf16 product.
// Weights and values.  The codes are the values, too: O^T[512 x NR] += codes^T (P scale), with the same tile read
// MN-major, accumulated in TMEM over the run's tiles of an item.  A position's scales are split as scale_b = m_b 2^e, e
// the exponent of the largest, and its weight is w = 2^(s + e - A), A an integer per row.  Block b's operand is
// w m_b 2^(A - R_b), R_b an integer per row and block, as two E4M3 terms: hi + lo, 8 significant bits, off by 2^-9 at
// most.  (w, m_b and the products are fp16 before: four roundings of 2^-11.)  Operands below 2^-6 are multiples of 2^-9,
// for 16 and 32 rows, whose lo has accumulators of its own and is held times 16, of 2^-13; there every position adds an
// offset of its own, spread evenly over +- half a step, before the rounding, so that many small weights keep their sum
// instead of all becoming 0 (0 stays 0).
//   R_b follows the largest operands that the tiles have in the block.  It puts them between 2^3.75 and 2^4.75 (2^6.75 and
// 2^7.75 where they rise), and moves when a tile's would lie above 2^8.75 or at or below 2^-0.25; the row's accumulators of
// the block are then scaled by a power of two, which is exact.  One R per block, because blocks differ: with one per row a
// block whose scales are 2^-9 of its neighbour's, or whose neighbour has a position of large weight, loses its bits to it.
// A block whose codes are all zero has no operand and counts for neither e nor R (the appends write a scale of 1 for it, far
// above ordinary ones); it has scores of 0 in every row, so its codes are looked at where the first two rows' are.  Moves
// cost: with a range of 4 instead of 8 powers of two 32 x 32768 positions of 64 heads (random queries and records) take
// 282 us instead of 240; one reference per row and one exponent per position, 220 us.  (R does not go further than 30 below
// its highest, nor 15 below A: what lies there is below 2^-30 of the row's largest operand in the block, or 2^-17 of
// its largest in any block, and the sums and factors stay finite.)
//   l = sum w 2^-e in fp32, out_b = O_b 2^(R_b - A) / l, lse = ln 2 (A + log2 l).
//
// What bounds it: HBM bytes (656 per position) for 16 rows; for more the steps of a tile inside an SM.  A tile of 64 rows
// takes 8000 cycles (4.2 us; an SM's share of the HBM rate is a tile per 1.9 us): shared memory feeds the tensor core for
// 3300 (M = 128 positions or dims, N = 64: 6 KB of operands per MMA of 32 dims or positions), and the softmax warps' steps
// follow one another: scores 1600 (with the waits for them), scales and rope 550, maxima 1200 (an SM reduces a value over a
// warp in 0.8 cycles: 1024 of them are 820), exchange 700, weights 350, operands 1400, their stores 900 (and 600 of waits
// for the PV, whose K slots come free one by one for the next tile's blocks).  Measured, 32 requests x 32768 positions: 64
// heads 241 us (2.9 TB/s), 32 heads 153 us (4.5 TB/s), 16 heads 126 us (5.5 TB/s); 1 x 8192 positions of 64 heads 19 us, 1
// x 77 of 16 heads 9.8 us.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <atomic>
#include <cstddef>

#include "smla_device.cuh"
#include "smla_internal.h"
#include "smla_ptx.cuh"
#include "smla_split_layout.cuh"

namespace smla {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kTopOperand = 8.75f;      // a (row, block)'s largest operand is at most 2^8.75, within E4M3's 448
constexpr float kWindow = 8.f;            // a reference moves when a tile's largest operand would lie further below that
constexpr float kLowest = 30.f;           // how far below its highest value a reference may go
constexpr float kAbove = 6.f;             // A is at most so far below the highest R: w m_b stay below 2^14.75, in fp16
constexpr float kSlack = 4.f;             // and moves when it is less far by more than this
constexpr float kFactor = 15.f;           // no R is further below A than this: 2^(A - R) stays in fp16
constexpr int kLeastExponent = -60;       // of the scale that a position counts with
constexpr int kMostTiles16 = 4, kMostTiles32 = 24;   // tiles of a CTA up to which row groups are of 16 and of 32

// Warps: the softmax warps (warp w: TMEM lanes of quadrant w % 4, row part w / 4), then one warp each for the
// copies, the QK and the PV, and one that describes the run for the merge.
enum { kCopyRole, kQkRole, kPvRole };

constexpr uint32_t kSlot = 16384;         // 128 positions x 128 bytes: one code block or the rope of a tile
constexpr int kChunks = 5;                // of a tile's scores: the four code blocks, then the rope
// Tiles between a tile's prefetch into L2 and its copy (32 x 32768 positions of 64 heads when a tile took 3.9 us: 249 us, 2
// tiles 253, 3 tiles 261, no prefetch 255).
constexpr int kAhead = 1;

template <int NR>
struct DC {
  static constexpr int kRing = NR == 64 ? 6 : NR == 32 ? 8 : 9;     // slots of code blocks
  static constexpr int kRopeSlots = NR == 16 ? 2 : 1;              // the rope's slot is free once its scores are done
  static constexpr int kScaleSlots = NR == 64 ? 1 : 3;
  static constexpr int kPBufs = NR == 64 ? 2 : 4;                   // weights of so many blocks
  static constexpr int kSBufs = 4;                                  // score accumulators
  // the maxima of a tile and of the next have places of their own where a warp may be a tile ahead of another: with the
  // weights of two blocks at a time the later ones wait for the PV of the first, so for every warp's
  static constexpr int kReds = kPBufs < 4 ? 1 : 2;
  // hi and lo terms (of q, and of the weights) meet in one accumulator for 64 rows, where TMEM is full; for fewer rows
  // they are one MMA of twice the columns and meet in the registers
  static constexpr int kPasses = NR == 64 ? 2 : 1;
  static constexpr int kOCols = NR == 64 ? NR : 2 * NR;             // columns of a block's O^T of one tile, or scores
  static constexpr float kLoUp = kPasses == 1 ? 16.f : 1.f;         // lo is stored times this
  // Row parts: 8 softmax warps.  (16, with half the rows per thread, take as long for 64 rows and longer for 32: 32 x
  // 32768 positions of 64 heads 231 us instead of 228.)
  static constexpr int kParts = 2;
  static constexpr int kSoftWarps = 4 * kParts;
  static constexpr int kThreads = 32 * (kSoftWarps + 4);
  // registers after setmaxnreg, of the 168 at launch: two warpgroups of 232 and one of 40 are 3 x 168
  static constexpr int kSoftRegs = 232, kMiscRegs = 40;
  static constexpr int HC = NR / kParts;       // rows of one softmax thread
  static constexpr uint32_t kQ8Chunk = 2 * NR * 128;
  static constexpr uint32_t kQ8 = 0;
  static constexpr uint32_t kQr = kQ8 + 4 * kQ8Chunk;
  static constexpr uint32_t kK = (kQr + NR * 128 + 1023) / 1024 * 1024;
  static constexpr int kPRow = 2 * NR;                            // bytes of a position's weights: hi, then lo
  static constexpr uint32_t kPBuf = 128 * kPRow;
  static constexpr uint32_t kRope = kK + kRing * kSlot;
  static constexpr uint32_t kP = kRope + kRopeSlots * kSlot;
  static constexpr uint32_t kScale = kP + kPBufs * kPBuf;
  static constexpr uint32_t kF = kScale + kScaleSlots * 2048;     // [2][NR] float
  static constexpr uint32_t kLen = kF + 2 * NR * 4;               // [2][NR] int
  static constexpr uint32_t kRed = kLen + 2 * NR * 4;             // [4 quadrants][NR][4 blocks] float
  static constexpr uint32_t kRow = kRed + kReds * 16 * NR * 4;  // per softmax warp [4 blocks][HC] 2^(A - R) fp16, [HC] -A
  static constexpr uint32_t kRowWarp = 4 * HC * 2 + HC * 4;
  static constexpr uint32_t kBar = kRow + kSoftWarps * kRowWarp;
  static constexpr uint32_t kBytes = kBar + 640;
  // TMEM: O^T of block b at kOCols b, score buffer i at kSCol + kOCols i
  static constexpr uint32_t kSCol = 4 * kOCols;
  static constexpr uint32_t kTmemCols = kSCol + kSBufs * kOCols;
  static_assert(kBytes <= 232448, "shared memory");
  static_assert(kTmemCols == 512 || kTmemCols == 256, "TMEM allocations are powers of two");
};

// Limits below this are meant to run out: nothing is issued and the call reports a timeout.
constexpr uint64_t kLeastWaitNs = 1000;

struct Bars {
  uint64_t kfull[9], kempty[9], rfull[2], rempty[2], sfull[4], sempty[4], scfull[3], scempty[3];
  uint64_t pfull[4], pempty[4], qfull, drain[2];
  uint32_t tmem;
  int abort;
  int armed_k[9], armed_r[2], armed_sc[3];            // copies armed so far per slot
  int pages_ok[3];                        // of the tile in each scale slot: bit h: page h is loaded
  int first_item, first_tile;             // this CTA's run of tiles [run_begin, run_end) of the batch
  int last_item, active;                  // its last item, the number of CTAs that have a run
  long long run_begin, run_end;
  long long units, last_begin, last_end;  // of the line that is shared out; its last item's tiles on it
};
static_assert(sizeof(Bars) <= 640, "barrier area");

// The barriers, one per lane: those that the softmax warps arrive on count these warps.
template <int kSoftWarps>
__device__ __forceinline__ void init_bars(Bars* bars, const DenseParams& p, int lane, const CUtensorMap* map,
                                          const CUtensorMap* smap) {
  constexpr int kBars = offsetof(Bars, tmem) / 8;
  constexpr uint64_t kBySoftmax = (15ull << offsetof(Bars, sempty) / 8) | (7ull << offsetof(Bars, scempty) / 8) |
                                  (15ull << offsetof(Bars, pfull) / 8) | (1ull << offsetof(Bars, qfull) / 8);
  static_assert(kBars <= 64, "one bit per barrier");
  for (int i = lane; i < kBars; i += 32)
    ptx::mbar_init(reinterpret_cast<uint64_t*>(bars) + i, kBySoftmax >> i & 1 ? kSoftWarps : 1);
  if (lane < 9) bars->armed_k[lane] = 0;
  if (lane < 2) bars->armed_r[lane] = 0;
  if (lane < 3) bars->armed_sc[lane] = 0;
  if (lane == 0) {
    bars->abort = p.wait_ns < kLeastWaitNs;
    ptx::prefetch_tensormap(map);
    ptx::prefetch_tensormap(smap);
  }
  ptx::fence_mbar_init();
}

// One (request, row group): rows row0 .. row0 + nrows - 1 of the request's s_q H rows.
struct Rows {
  int req, row0, nrows;
};

__device__ __forceinline__ Rows rows_of(const DenseParams& p, int i) {
  Rows r;
  r.req = i / p.groups;
  r.row0 = (i - r.req * p.groups) * p.nr;
  r.nrows = min(p.nr, p.q_per_req * p.H - r.row0);
  return r;
}

__device__ __forceinline__ int clamped_len(const DenseParams& p, int b) {
  const long long table = (long long)p.max_pages * kPageSize;
  const long long n = max(__ldg(p.seq_lens + b), 0);
  return (int)min(n, table);
}

// Lengths of an item's queries (clamped to [0, table]) and its tiles: at least 1, so that a group without
// positions has one empty tile.
struct Lens {
  int max_len, min_len, tiles;
};

__device__ __forceinline__ Lens lens_of(const DenseParams& p, const Rows& r) {
  Lens n{0, 0x7fffffff, 0};
  int b = r.req * p.q_per_req + r.row0 / p.H;
  const int last = r.req * p.q_per_req + (r.row0 + r.nrows - 1) / p.H;
#pragma unroll 1
  for (; b <= last; ++b) {
    const int len = clamped_len(p, b);
    n.max_len = max(n.max_len, len);
    n.min_len = min(n.min_len, len);
  }
  n.tiles = max(1, (int)(((long long)n.max_len + kDenseTile - 1) / kDenseTile));
  return n;
}

// First unit of CTA c's run when T units are shared out over n CTAs.
__device__ __forceinline__ long long run_start(long long T, int n, int c) {
  const unsigned long long x = (unsigned long long)T * c;
  return x >> 32 ? x / n : (uint32_t)x / (uint32_t)n;
}

// What the kernel leaves for the merge: the item that begins in a CTA's run and ends in a later one's, if any, and
// the number of runs that it crosses (0: nothing to join).
struct RunDesc {
  int item, parts;
};

// Walks the (item, tile) pairs of a run; every role has its own:  while (w.here(p)) { ...; w.next(); }
struct Walk {
  int i, t, left;
  bool entered = false;
  Lens n;
  __device__ __forceinline__ explicit Walk(const Bars* bars)
      : i(bars->first_item), t(bars->first_tile), left((int)(bars->run_end - bars->run_begin)) {}
  __device__ __forceinline__ bool here(const DenseParams& p) {
    if (left > 0 && !entered) {
      n = lens_of(p, rows_of(p, i));
      entered = true;
    }
    return left > 0;
  }
  __device__ __forceinline__ bool last_of_segment() const { return left == 1 || t == n.tiles - 1; }
  __device__ __forceinline__ void next() {
    --left;
    if (++t == n.tiles) {
      t = 0;
      ++i;
      entered = false;
    }
  }
};

// A ring position: slot and the parity of its current use.
template <int N>
struct Ring {
  int slot = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next() {
    if (++slot == N) {
      slot = 0;
      parity ^= 1;
    }
  }
};

// A wait for a slot to be freed (the other parity) passes at once on the ring's first round: an mbarrier that has
// completed no phase yet reports the phase before its first as complete.
// A wait of a whole warp, bounded by p.wait_ns.  The common case is one try; once a wait has given up (ok 0) a
// role runs its loop to the end without arriving or issuing, so that the named barriers of the softmax warps stay
// matched.  (`ok` passes through an empty asm: otherwise the compiler makes a copy of the rest of the role for
// each wait that may give up.)
#define SMLA_WAIT(bar, par)                                                                               \
  do {                                                                                                    \
    if (__builtin_expect(__any_sync(0xffffffffu, !ptx::mbar_try_wait((bar), (par))), 0)) {                \
      if (ok) ok = ptx::mbar_wait_rest((bar), (par), &bars->abort, p.wait_ns);                            \
      asm volatile("" : "+r"(ok));                                                                        \
    }                                                                                                     \
  } while (0)

// ----------------------------------------------------------------------------- copies

__device__ __forceinline__ int page_entry(const DenseParams& p, int req, int max_len, int lp) {
  return lp < p.max_pages && (long long)lp * kPageSize < max_len
             ? __ldg(p.block_table + (size_t)req * p.max_pages + lp)
             : -1;
}

template <int NR>
__device__ void copy_role(const DenseParams& p, const CUtensorMap* map, const CUtensorMap* smap, uint32_t base,
                          Bars* bars, int lane) {
  using C = DC<NR>;
  Walk w(bars);
  int req = 0;
  Ring<C::kRing> k;
  Ring<C::kScaleSlots> sc;
  Ring<C::kRopeSlots> rope;
  uint32_t ok = p.wait_ns >= kLeastWaitNs;
  // block-table entries of 16 tiles per load, one lane each, the next 16 tiles' already in flight
  int cur = 0, nxt = 0, base_lp = 0, item = -1;
#pragma unroll 1
  while (w.here(p)) {
    const int lp = 2 * w.t;
    const bool enters = item != w.i;
    if (enters) {
      item = w.i;
      const Rows r = rows_of(p, item);
      req = r.req;
      base_lp = lp;
      nxt = page_entry(p, req, w.n.max_len, lp + lane);
      if (lane == 0) {
        const int last = req * p.q_per_req + (r.row0 + r.nrows - 1) / p.H;
#pragma unroll 1
        for (int b = req * p.q_per_req + r.row0 / p.H; b <= last; ++b)
          if (__ldg(p.seq_lens + b) > (long long)p.max_pages * kPageSize) atomicOr(p.err, SMLA_DEVERR_PAGE_RANGE);
      }
    }
    if (enters || lp == base_lp + 32) {
      base_lp = lp;
      cur = nxt;
      nxt = page_entry(p, req, w.n.max_len, lp + 32 + lane);
    }
    const int pg[2] = {__shfl_sync(0xffffffffu, cur, lp - base_lp), __shfl_sync(0xffffffffu, cur, lp - base_lp + 1)};
    int good = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool used = (long long)(lp + h) * kPageSize < w.n.max_len;
      const bool in_cache = pg[h] >= 0 && (int64_t)pg[h] < p.num_pages;
      if (used && in_cache) good |= 1 << h;
      if (used && !in_cache && lane == 0) atomicOr(p.err, SMLA_DEVERR_PAGE_RANGE);
    }
    const uint32_t n_good = (good & 1) + (good >> 1);
    // a later tile of the item into L2: K slots come free one by one behind the PV, and their loads would bring the
    // latency of HBM into every tile
    const int ahead = lp - base_lp + 2 * kAhead + (lane & 1);
    const int page_cur = __shfl_sync(0xffffffffu, cur, ahead & 31), page_nxt = __shfl_sync(0xffffffffu, nxt, ahead & 31);
    const int page = ahead < 32 ? page_cur : page_nxt;
    if (w.left > kAhead && lane < 2 && page >= 0 && (int64_t)page < p.num_pages)
      ptx::prefetch_l2_bulk(p.kv + (size_t)page * kPageSize * kRecordBytes, kPageSize * kRecordBytes);
    SMLA_WAIT(&bars->scempty[sc.slot], sc.parity ^ 1);
    if (ok && ptx::elect_one()) {
      bars->pages_ok[sc.slot] = good;
      ++bars->armed_sc[sc.slot];
      ptx::mbar_arrive_expect_tx(&bars->scfull[sc.slot], n_good * 1024);
      for (int h = 0; h < 2; ++h)
        if (good >> h & 1)
          ptx::tma_load_3d(base + C::kScale + sc.slot * 2048 + h * 1024, smap, kDLatent, 0, pg[h],
                           &bars->scfull[sc.slot]);
    }
    __syncwarp();
    sc.next();
    // the rope between the blocks that are loaded ahead and those that wait for the PV of the tile before
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      if (c == 2) {
        SMLA_WAIT(&bars->rempty[rope.slot], rope.parity ^ 1);
        if (ok && ptx::elect_one()) {
          ++bars->armed_r[rope.slot];
          ptx::mbar_arrive_expect_tx(&bars->rfull[rope.slot], n_good * (kSlot / 2));
          for (int h = 0; h < 2; ++h)
            if (good >> h & 1)
              ptx::tma_load_3d(base + C::kRope + rope.slot * kSlot + h * (kSlot / 2), map, kDLatent + 16, 0, pg[h],
                               &bars->rfull[rope.slot]);
        }
        __syncwarp();
        rope.next();
      }
      SMLA_WAIT(&bars->kempty[k.slot], k.parity ^ 1);
      if (ok && ptx::elect_one()) {
        ++bars->armed_k[k.slot];
        ptx::mbar_arrive_expect_tx(&bars->kfull[k.slot], n_good * (kSlot / 2));
        for (int h = 0; h < 2; ++h)
          if (good >> h & 1)
            ptx::tma_load_3d(base + C::kK + k.slot * kSlot + h * (kSlot / 2), map, 128 * c, 0, pg[h],
                             &bars->kfull[k.slot]);
      }
      __syncwarp();
      k.next();
    }
    w.next();
  }
}

// After a wait that gave up: every copy that was armed has to land before the CTA leaves.  Nothing arms a slot
// again by then, so the slot's last phase is waited for.
__device__ void drain_copies(uint64_t* bar, const int* armed, int n, int lane) {
  int never = 0;
  for (int s = 0; s < n; ++s)
    if (armed[s] > 0) ptx::mbar_wait_warp(&bar[s], (uint32_t)(armed[s] - 1) & 1u, &never, lane, 100000000ull);
}

// ----------------------------------------------------------------------------- MMA issue

template <int NR>
__device__ void qk_role(const DenseParams& p, uint32_t base, uint32_t tmem, Bars* bars, int lane) {
  using C = DC<NR>;
  constexpr uint32_t kIdescCodes = ptx::idesc_e4m3(128, C::kOCols), kIdescRope = ptx::idesc_bf16(128, NR);
  Walk w(bars);
  Ring<C::kRing> k;
  Ring<C::kSBufs> s;
  Ring<C::kRopeSlots> rope;
  uint32_t qpar = 0;
  uint32_t ok = p.wait_ns >= kLeastWaitNs;
  int item = -1;
  const uint64_t dq = ptx::sw128_desc(base + C::kQ8, 16, 1024), dr = ptx::sw128_desc(base + C::kQr, 16, 1024);
#pragma unroll 1
  while (w.here(p)) {
    if (item != w.i) {
      item = w.i;
      SMLA_WAIT(&bars->qfull, qpar);
      qpar ^= 1;
    }
#pragma unroll 1
    for (int c = 0; c < kChunks; ++c) {
      SMLA_WAIT(&bars->sempty[s.slot], s.parity ^ 1);
      SMLA_WAIT(c < 4 ? &bars->kfull[k.slot] : &bars->rfull[rope.slot], c < 4 ? k.parity : rope.parity);
      ptx::tc_fence_after();
      const uint32_t ks = k.slot, d = tmem + C::kSCol + C::kOCols * s.slot, cu = c;
      if (ok && ptx::elect_one()) {
        if (c == 4) {
          const uint64_t dk = ptx::sw128_desc(base + C::kRope + rope.slot * kSlot, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) ptx::mma_f16_ss(d, dk + 2 * kk, dr + 2 * kk, kIdescRope, kk > 0);
          ptx::mma_commit(&bars->rempty[rope.slot]);     // (the codes stay for the PV)
        } else {
          const uint64_t dk = ptx::sw128_desc(base + C::kK + ks * kSlot, 16, 1024);
          const uint64_t dqb = dq + (uint64_t)((cu * C::kQ8Chunk) >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
#pragma unroll
            for (int pass = 0; pass < C::kPasses; ++pass)
              ptx::mma_f8_ss(d, dk + 2 * kk, dqb + 2 * kk + (uint64_t)((pass * NR * 128) >> 4), kIdescCodes,
                             kk > 0 || pass > 0);
        }
        ptx::mma_commit(&bars->sfull[s.slot]);
      }
      __syncwarp();
      if (c < 4) k.next();
      s.next();
    }
    rope.next();
    w.next();
  }
  if (ptx::elect_one()) ptx::mma_commit(&bars->drain[0]);
  __syncwarp();
}

template <int NR>
__device__ void pv_role(const DenseParams& p, uint32_t base, uint32_t tmem, Bars* bars, int lane) {
  using C = DC<NR>;
  constexpr int N = C::kOCols;
  constexpr uint32_t kIdesc = ptx::idesc_e4m3(128, N) | (1u << 15) | (1u << 16);     // A and B MN-major
  Walk w(bars);
  Ring<C::kRing> k;
  Ring<C::kPBufs> pb;
  uint32_t ok = p.wait_ns >= kLeastWaitNs;
  int item = -1;
#pragma unroll 1
  while (w.here(p)) {
    const uint32_t more = item == w.i;                    // not the segment's first tile
    item = w.i;
#pragma unroll 1
    for (int b = 0; b < 4; ++b) {
      SMLA_WAIT(&bars->pfull[pb.slot], pb.parity);
      ptx::tc_fence_after();
      const uint32_t ks = k.slot, ps = pb.slot, d = tmem + N * b;
      if (ok && ptx::elect_one()) {
        // codes^T: 128-byte rows of one position, 8-position groups 1024 bytes apart; 32 positions per MMA
        const uint64_t dv = ptx::sw128_desc(base + C::kK + ks * kSlot, 1024, 1024);
        const uint64_t dp = ptx::swz_desc(base + C::kP + ps * C::kPBuf, 8 * C::kPRow, 8 * C::kPRow, C::kPRow);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
#pragma unroll
          for (int pass = 0; pass < C::kPasses; ++pass)
            ptx::mma_f8_ss(d, dv + (uint64_t)(256 * kk),
                           dp + (uint64_t)((32 * C::kPRow * kk + NR * pass) >> 4), kIdesc,
                           kk > 0 || pass > 0 ? 1 : more);
        ptx::mma_commit(&bars->kempty[k.slot]);
        ptx::mma_commit(&bars->pempty[pb.slot]);
      }
      __syncwarp();
      k.next();
      pb.next();
    }
    w.next();
  }
  if (ptx::elect_one()) ptx::mma_commit(&bars->drain[1]);
  __syncwarp();
}

// ----------------------------------------------------------------------------- softmax

// Reduce v[N] over the warp's lanes with op; lane i ends with the result of element i % N.
template <int N, typename Op>
__device__ __forceinline__ float reduce_scatter(float (&v)[N], int lane, Op op) {
#pragma unroll
  for (int h = N / 2; h >= 1; h >>= 1) {
    const bool up = lane & h;
#pragma unroll
    for (int i = 0; i < h; ++i) {
      const float send = up ? v[i] : v[i + h];
      const float got = __shfl_xor_sync(0xffffffffu, send, h);
      v[i] = op(up ? v[i + h] : v[i], got);
    }
  }
  float r = v[0];
#pragma unroll
  for (int h = N; h < 32; h <<= 1) r = op(r, __shfl_xor_sync(0xffffffffu, r, h));
  return r;
}

__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// Rows of one item into the Q operands: hi and lo E4M3 codes of the latent part scaled by 2^-x, the rope as it is;
// each row's factor 2^x sm_scale log2 e and length go to buffer `buf`.
template <int NR>
__device__ __forceinline__ void load_q(const DenseParams& p, int item, unsigned char* sm, uint32_t base, int buf,
                                       int warp, int lane) {
  using C = DC<NR>;
  constexpr int kRows = NR / C::kSoftWarps;             // rows warp, warp + kSoftWarps, ... of this warp
  const Rows it = rows_of(p, item);
  float* f = reinterpret_cast<float*>(sm + C::kF) + buf * NR;
  int* lens = reinterpret_cast<int*>(sm + C::kLen) + buf * NR;
  const float kf = p.sm_scale * kLog2e;
  const uint16_t* q0 = p.q + ((size_t)it.req * p.q_per_req * p.H + it.row0) * kDQK;
  const int b = lane >> 3, u = lane & 7;
  uint4 raw[kRows][2], rope[(kRows + 3) / 4];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = warp + C::kSoftWarps * i;
    const uint4* src = reinterpret_cast<const uint4*>(q0 + (size_t)r * kDQK);
    raw[i][0] = raw[i][1] = make_uint4(0u, 0u, 0u, 0u);
    if (r < it.nrows) {
      raw[i][0] = __ldg(src + 2 * lane);
      raw[i][1] = __ldg(src + 2 * lane + 1);
    }
  }
  // the rope, 16 bytes per lane: four rows at a time
#pragma unroll
  for (int i = 0; i < (kRows + 3) / 4; ++i) {
    const int k = 4 * i + b, r = warp + C::kSoftWarps * k;
    rope[i] = make_uint4(0u, 0u, 0u, 0u);
    if (k < kRows && r < it.nrows) rope[i] = __ldg(reinterpret_cast<const uint4*>(q0 + (size_t)r * kDQK) + 64 + u);
  }
  if (lane < kRows) {
    const int r = warp + C::kSoftWarps * lane;
    lens[r] = r < it.nrows ? clamped_len(p, it.req * p.q_per_req + (it.row0 + r) / p.H) : 0x7fffffff;
  }
#pragma unroll
  for (int i = 0; i < (kRows + 3) / 4; ++i) {
    const int k = 4 * i + b;
    if (k < kRows) ptx::sts128(base + C::kQr + swz128(warp + C::kSoftWarps * k, u), rope[i]);
  }
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int r = warp + C::kSoftWarps * k;
    const uint32_t wds[8] = {raw[k][0].x, raw[k][0].y, raw[k][0].z, raw[k][0].w,
                             raw[k][1].x, raw[k][1].y, raw[k][1].z, raw[k][1].w};
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(wds[i] << 16)), fabsf(__uint_as_float(wds[i] & 0xffff0000u))));
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    // x = floor(log2 amax) - 7, kept where 2^x and 2^-x are normal floats
    const int x = amax > 0.f ? min(max((int)(__float_as_uint(amax) >> 23) - 127 - 7, -120), 120) : 0;
    const float down = exp2_int(-x);
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint16_t h2[2], l2[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float a = __uint_as_float(wds[2 * i + j] << 16) * down, c = __uint_as_float(wds[2 * i + j] & 0xffff0000u) * down;
        a = isinf(a) ? CUDART_NAN_F : a;                 // an infinite q makes the row NaN
        c = isinf(c) ? CUDART_NAN_F : c;
        h2[j] = f32x2_to_e4m3x2(a, c);
        const float2 back = f16x2_to_f32x2(e4m3x2_to_f16x2(h2[j]));
        l2[j] = f32x2_to_e4m3x2(a - back.x, c - back.y);
      }
      hi[i] = (uint32_t)h2[0] | ((uint32_t)h2[1] << 16);
      lo[i] = (uint32_t)l2[0] | ((uint32_t)l2[1] << 16);
    }
    const uint32_t q8 = base + C::kQ8 + b * C::kQ8Chunk;
    ptx::sts128(q8 + swz128(r, u), make_uint4(hi[0], hi[1], hi[2], hi[3]));
    ptx::sts128(q8 + swz128(NR + r, u), make_uint4(lo[0], lo[1], lo[2], lo[3]));
    if (lane == 0) f[r] = exp2_int(x) * kf;
  }
}

template <int NR>
__device__ __forceinline__ void tmem_st(uint32_t a, const uint32_t (&r)[NR]) {
  if constexpr (NR == 32) ptx::tmem_st32(a, r);
  else if constexpr (NR == 16) ptx::tmem_st16(a, r);
  else ptx::tmem_st8(a, r);
}
template <int NR>
__device__ __forceinline__ void tmem_ld(uint32_t a, uint32_t (&r)[NR]) {
  if constexpr (NR == 32) ptx::tmem_ld32(a, r);
  else if constexpr (NR == 16) ptx::tmem_ld16(a, r);
  else ptx::tmem_ld8(a, r);
}
// The exponent e that a position's weights take from its scales.
__device__ __forceinline__ int scale_exponent(const float4& s) {
  const float top = fmaxf(fmaxf(fabsf(s.x), fabsf(s.y)), fmaxf(fabsf(s.z), fabsf(s.w)));
  return min(max((int)(__float_as_uint(top) >> 23) - 127, kLeastExponent), 126);
}

// Two fp16 pairs -> four E4M3 codes in one word (round to nearest even, saturating), and back.
__device__ __forceinline__ uint32_t f16x4_to_e4m3x4(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("{\n .reg .b16 x, y;\n cvt.rn.satfinite.e4m3x2.f16x2 x, %1;\n cvt.rn.satfinite.e4m3x2.f16x2 y, %2;\n"
      " mov.b32 %0, {x, y};\n}\n"
      : "=r"(r)
      : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t w, uint32_t& a, uint32_t& b) {
  asm("{\n .reg .b16 x, y;\n mov.b32 {x, y}, %2;\n cvt.rn.f16x2.e4m3x2 %0, x;\n cvt.rn.f16x2.e4m3x2 %1, y;\n}\n"
      : "=r"(a), "=r"(b)
      : "r"(w));
}
__device__ __forceinline__ __half2 as_half2(uint32_t v) { return *reinterpret_cast<const __half2*>(&v); }
__device__ __forceinline__ uint32_t as_u32(__half2 v) { return *reinterpret_cast<const uint32_t*>(&v); }

// Makes the codes of positions that some row does not see harmless for the PV (a weight of 0 must give 0):
// NaN codes become 0, and every code of a position that no row sees.  (A row that does see a NaN code has a NaN
// score, so it is NaN whatever the value.)  The threads of a row part take every kParts-th block.
template <int NR>
__device__ __noinline__ void clean_codes(uint32_t base, int slot, int tok, int part, bool seen) {
  using C = DC<NR>;
#pragma unroll 1
  for (int b = 0; b < 4; ++b) {
    if (b % C::kParts == part) {
      const uint32_t at = base + C::kK + slot * kSlot;
#pragma unroll 1
      for (int u = 0; u < 8; ++u) {
        uint4 v = ptx::lds128(at + swz128(tok, u));
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = seen ? w[i] & ~__vcmpeq4(w[i] & 0x7f7f7f7fu, 0x7f7f7f7fu) : 0u;
        ptx::sts128(at + swz128(tok, u), make_uint4(w[0], w[1], w[2], w[3]));
      }
    }
    if (++slot == C::kRing) slot = 0;
  }
}

// Which of the blocks in `maybe` hold codes of zero alone at position tok.  (Another row part may be cleaning the codes of
// a position at the same time: of one that no row sees, whose weights are 0, or NaN codes, whose scores are never 0.)
template <int NR>
__device__ __noinline__ uint32_t zero_blocks(uint32_t base, int slot, int tok, uint32_t maybe) {
  using C = DC<NR>;
#pragma unroll 1
  for (int b = 0; b < 4; ++b) {
    if (maybe >> b & 1) {
      const uint32_t at = base + C::kK + slot * kSlot;
      uint32_t any = 0;
#pragma unroll 1
      for (int u = 0; u < 8 && any == 0; ++u) {
        const uint4 v = ptx::lds128(at + swz128(tok, u));
        any = (v.x | v.y | v.z | v.w) & 0x7f7f7f7fu;
      }
      if (any) maybe &= ~(1u << b);
    }
    if (++slot == C::kRing) slot = 0;
  }
  return maybe;
}

// A scale as the values' operands take it: 0 for a block without values, or a NaN or infinite one (whose rows are NaN
// by their scores).
__device__ __forceinline__ float value_scale(float s, bool zero) { return !zero && fabsf(s) < CUDART_INF_F ? s : 0.f; }

// v[lane % N], of values that are the same in every lane: N - 1 selects.
template <int N>
__device__ __forceinline__ float pick(const float (&v)[N], int lane) {
  if constexpr (N == 1) {
    return v[0];
  } else {
    float h[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) h[i] = lane & (N / 2) ? v[i + N / 2] : v[i];
    return pick<N / 2>(h, lane);
  }
}

// One dim of a block for HC rows (pairs), times the rows' factors, out to global memory: lanes 2j, 2j + 1 hold dims
// d, d + 1 of two rows; the first ends with both dims of the first row, the other (`second`) with both of the second,
// and stores them at `to` (rows 2 apart; `left` of them from this thread's first on), as bf16 or fp32.
template <int HC, bool kBf16>
__device__ __forceinline__ void write_block(const uint64_t (&x)[HC / 2], uint32_t row_c, int left, bool second, void* to) {
#pragma unroll
  for (int i = 0; i < HC / 2; i += 2) {
    const ulonglong2 f = ptx::lds128_pairs(row_c + i * 8);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float2 v = ptx::unpack2(ptx::mul2(x[i + j], j ? f.y : f.x));
      const float got = __shfl_xor_sync(0xffffffffu, second ? v.x : v.y, 1);
      const float d0 = second ? got : v.x, d1 = second ? v.y : got;
      if (2 * (i + j) < left) {
        const int at = 2 * (i + j) * kDLatent;
        if constexpr (kBf16) *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(to) + at) = f32x2_to_bf16x2(d0, d1);
        else *reinterpret_cast<float2*>(static_cast<float*>(to) + at) = make_float2(d0, d1);
      }
    }
  }
}

template <int NR>
__device__ void softmax_role(const DenseParams& p, unsigned char* sm, uint32_t base, uint32_t tmem, Bars* bars, int warp,
                             int lane, float* o_part, float* lse_part) {
  using C = DC<NR>;
  constexpr int HC = C::HC;                             // rows per thread
  constexpr int kChunk = 8;                             // rows that are scaled back or written at once
  const int part = warp >> 2, quad = warp & 3, col0 = part * HC;
  const int tok = 32 * quad + lane;
  const uint32_t lane_base = tmem + ((uint32_t)(32 * quad) << 16);
  const float kf = p.sm_scale * kLog2e;
  const uint32_t row_c = base + C::kRow + warp * C::kRowWarp, row_na = row_c + 4 * HC * 2;
  Walk w(bars);
  Ring<C::kSBufs> s;
  Ring<C::kScaleSlots> sc;
  Ring<C::kPBufs> pb;
  int kslot = 0;
  uint32_t red = base + C::kRed + col0 * 16;            // values of a part's rows meet here, [quad][row][block]
  const uint32_t fac = red;                             // and their factors, [block][row], in the first quadrant's place
  uint32_t last_par = 0;                                // of the last tile's last PV
  uint32_t ok = p.wait_ns >= kLeastWaitNs;
  bool first = true, begins = w.t == 0;
  int buf = 0;
  uint64_t l[HC / 2];                                   // row sums over this thread's positions, pairs of rows
  // Lane l keeps references of row col0 + l % HC: R of blocks kRefs (l / HC) + j (NaN while no value of the block was
  // met), their highest values, and A (NaN while the row has met no position).  Every warp of the part keeps the same.
  constexpr int kRefs = HC / 8;
  const int row = lane % HC, block0 = lane / HC * kRefs;
  float ref[kRefs], top[kRefs], level = CUDART_NAN_F;
  float upper[kRefs], lower[kRefs];                     // a reference stays for a largest operand up to, and above, these
#pragma unroll
  for (int j = 0; j < kRefs; ++j) ref[j] = CUDART_NAN_F, top[j] = 0.f, upper[j] = lower[j] = -CUDART_INF_F;
  bool live = false;                                    // the part has rows

  // every PV of the tiles before is done: their accumulators (dims 128 b + tok) can be read and scaled
  auto wait_pv = [&]() {
    SMLA_WAIT(&bars->pempty[3 % C::kPBufs], last_par);
    ptx::tc_fence_after();
  };
  int item = -1, done = -1;                             // items whose rows are loaded, whose segment has ended
  bool whole = false;                                   // the segment is its whole item
#pragma unroll 1
  for (;;) {
    const bool more = w.here(p);
    if (more && item != w.i) {
      // the next item's rows, so that its scores can start beside the last one's PV
      done = item;
      item = w.i;
      buf ^= 1;
      live = col0 < rows_of(p, item).nrows;
      load_q<NR>(p, item, sm, base, buf, warp, lane);
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (ok && lane == 0) ptx::mbar_arrive(&bars->qfull);
    }
    if (!more) done = item;
    if (first && done >= 0) {
      const Rows it = rows_of(p, done);
      // row sums over the 128 positions of the tiles
      float ls[HC];
#pragma unroll
      for (int i = 0; i < HC / 2; ++i) {
        const float2 x = ptx::unpack2(l[i]);
        ls[2 * i] = x.x;
        ls[2 * i + 1] = x.y;
      }
      const float sum = reduce_scatter<HC>(ls, lane, [](float a, float b) { return a + b; });
      if (lane < HC) ptx::sts32f(red + (quad * NR + lane) * 16, sum);
      ptx::named_bar_sync(1 + part, 128);
      // a run's first segment that continues an item goes to slot 0 of the CTA, its last segment to slot 1
      const size_t slot = 2 * (size_t)blockIdx.x + (begins ? 1 : 0);
      float factor = 0.f;                                 // of block `quad`
      {
        const uint32_t at = red + row * 16;
        const float z = (ptx::lds32f(at) + ptx::lds32f(at + NR * 16)) +
                        (ptx::lds32f(at + 2 * NR * 16) + ptx::lds32f(at + 3 * NR * 16));
        const bool none = z == 0.f && !(level == level);   // (a sum of 0 beside positions is refused as a NaN)
        int ez;
        const float mz = frexpf(z, &ez);                  // (the exponents meet as whole numbers)
        const float lse = none ? -CUDART_INF_F : z == 0.f ? CUDART_NAN_F : (log2f(mz) + ((float)ez + level)) * kLn2;
        if (quad == 0 && lane < HC && ok && col0 + lane < it.nrows) {
          if (whole) p.lse[(size_t)it.req * p.q_per_req * p.H + it.row0 + col0 + lane] = lse;
          else lse_part[slot * NR + col0 + lane] = lse;
        }
        // 2^(R - A) / l, by which a block's accumulators become outputs
#pragma unroll
        for (int j = 0; j < kRefs; ++j) {
          if (block0 + j != quad) continue;
          float inv = none ? 0.f : CUDART_NAN_F;
          if (z > 0.f) inv = ref[j] == ref[j] ? ldexpf(1.f / mz, (int)fminf(fmaxf(ref[j] - level, -400.f), 400.f) - ez) : 0.f;
          factor = inv;
        }
      }
      ptx::named_bar_sync(1 + part, 128);
      if (block0 <= quad && quad < block0 + kRefs) ptx::sts32f(fac + (quad * HC + row) * 4, factor);
      ptx::named_bar_sync(1 + part, 128);
      // lanes 2j, 2j + 1 hold dims d, d + 1 of two rows: the first ends with both dims of the first row, the other
      // with both of the second, and writes them there
      const bool second = lane & 1;
      const int c0 = col0 + (second ? 1 : 0);             // this thread's rows: c0, c0 + 2, ...
      const size_t row0 = whole ? (size_t)it.req * p.q_per_req * p.H + it.row0 : slot * NR;
      const size_t at = (row0 + c0) * kDLatent + (tok & ~1);
      const int rows_left = ok ? it.nrows - c0 : 0;
      wait_pv();
#pragma unroll 1
      for (int i0 = 0; i0 < HC; i0 += kChunk) {
        uint32_t hi[4][kChunk], lo[4][kChunk];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          tmem_ld<kChunk>(lane_base + C::kOCols * b + col0 + i0, hi[b]);
          if constexpr (C::kPasses == 1) tmem_ld<kChunk>(lane_base + C::kOCols * b + NR + col0 + i0, lo[b]);
        }
        ptx::tmem_wait_ld();
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          uint64_t x[kChunk / 2];
#pragma unroll
          for (int i = 0; i < kChunk / 2; ++i) {
            x[i] = ptx::pack2(hi[b][2 * i], hi[b][2 * i + 1]);
            if constexpr (C::kPasses == 1)
              x[i] = ptx::fma2(ptx::pack2(lo[b][2 * i], lo[b][2 * i + 1]), ptx::pack2(1.f / C::kLoUp, 1.f / C::kLoUp), x[i]);
          }
          const size_t to = at + 128 * b + (size_t)i0 * kDLatent;
          const uint32_t by = fac + (b * HC + i0) * 4;
          if (whole) write_block<kChunk, true>(x, by, rows_left - i0, second, p.out + to);
          else write_block<kChunk, false>(x, by, rows_left - i0, second, o_part + to);
        }
      }
      ptx::tc_fence_before();
      begins = true;
    }
    if (!more) break;
    if (first) {
      ptx::named_bar_sync(1 + C::kParts, C::kSoftWarps * 32);   // the rows' factors and lengths are written
#pragma unroll
      for (int i = 0; i < HC / 2; ++i) l[i] = 0;
#pragma unroll
      for (int j = 0; j < kRefs; ++j) ref[j] = CUDART_NAN_F, upper[j] = lower[j] = -CUDART_INF_F;
      level = CUDART_NAN_F;
    }
    // scores of this thread's position for its HC rows, in units of log2
    SMLA_WAIT(&bars->scfull[sc.slot], sc.parity);
    const float4 s4 = ptx::lds128f(base + C::kScale + sc.slot * 2048 + tok * 16);
    const int pages = bars->pages_ok[sc.slot];
    __syncwarp();
    if (ok && lane == 0) ptx::mbar_arrive(&bars->scempty[sc.slot]);
    sc.next();
    uint64_t acc[HC / 2];                               // pairs of rows
    uint32_t zero = 0;                                  // bit b: the position may have no value in block b
    {
      float4 rot = s4;
#pragma unroll
      for (int i = 0; i < HC / 2; ++i) acc[i] = 0;
      // two blocks at a time: their TMEM loads wait once
#pragma unroll 1
      for (int b = 0; b < 4; b += 2) {
        const uint32_t a0 = lane_base + C::kSCol + C::kOCols * s.slot + col0;
        const int s0 = s.slot;
        SMLA_WAIT(&bars->sfull[s.slot], s.parity);
        s.next();
        const uint32_t a1 = lane_base + C::kSCol + C::kOCols * s.slot + col0;
        const int s1 = s.slot;
        SMLA_WAIT(&bars->sfull[s.slot], s.parity);
        s.next();
        ptx::tc_fence_after();
        const uint64_t scale0 = ptx::pack2(rot.x, rot.x), scale1 = ptx::pack2(rot.y, rot.y);
        rot = make_float4(rot.z, rot.w, rot.x, rot.y);
        uint32_t x0[HC], y0[HC], x1[HC], y1[HC];
        tmem_ld<HC>(a0, x0);
        if constexpr (C::kPasses == 1) tmem_ld<HC>(a0 + NR, y0);
        tmem_ld<HC>(a1, x1);
        if constexpr (C::kPasses == 1) tmem_ld<HC>(a1 + NR, y1);
        ptx::tmem_wait_ld();
        if (((x0[0] | x0[1]) & 0x7fffffffu) == 0) zero |= 1u << b;
        if (((x1[0] | x1[1]) & 0x7fffffffu) == 0) zero |= 2u << b;
#pragma unroll
        for (int i = 0; i < HC; i += 2) {
          uint64_t x = ptx::pack2(x0[i], x0[i + 1]), y = ptx::pack2(x1[i], x1[i + 1]);
          if constexpr (C::kPasses == 1) {
            x = ptx::add2(x, ptx::pack2(y0[i], y0[i + 1]));
            y = ptx::add2(y, ptx::pack2(y1[i], y1[i + 1]));
          }
          acc[i / 2] = ptx::fma2(y, scale1, ptx::fma2(x, scale0, acc[i / 2]));
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (ok && lane == 0) {
          ptx::mbar_arrive(&bars->sempty[s0]);
          ptx::mbar_arrive(&bars->sempty[s1]);
        }
      }
    }
    // the scales that the position's values have: a block without values has none
    if (__builtin_expect(zero != 0, 0)) zero = live ? zero_blocks<NR>(base, kslot, tok, zero) : 0u;
    const float4 v4 = make_float4(value_scale(s4.x, zero & 1), value_scale(s4.y, zero & 2), value_scale(s4.z, zero & 4),
                                  value_scale(s4.w, zero & 8));
    const int e = scale_exponent(v4);
    float4 lg;                                          // log2(scale_b 2^-e)
    {
      const float d = exp2_int(-e);
      lg = make_float4(ptx::lg2_approx(fabsf(v4.x * d)), ptx::lg2_approx(fabsf(v4.y * d)), ptx::lg2_approx(fabsf(v4.z * d)),
                       ptx::lg2_approx(fabsf(v4.w * d)));
      // (a position with next to no value counts all the same, so that its weight is a float)
      if (e == kLeastExponent) lg.x = fmaxf(lg.x, 0.f);
    }
    __syncwarp();
    // s + e in powers of two: 2^x sm_scale log2 e (latent part) + (rope part sm_scale log2 e + e)
    SMLA_WAIT(&bars->sfull[s.slot], s.parity);
    ptx::tc_fence_after();
    {
      const uint32_t a = lane_base + C::kSCol + C::kOCols * s.slot + col0;
      const uint64_t kf2 = ptx::pack2(kf, kf), e2 = ptx::pack2((float)e, (float)e);
      const uint32_t fa = base + C::kF + (buf * NR + col0) * 4;
      uint32_t r[HC];
      tmem_ld<HC>(a, r);
      ptx::tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < HC; i += 4) {
        const ulonglong2 f = ptx::lds128_pairs(fa + i * 4);
        uint64_t* d = &acc[i / 2];
        d[0] = ptx::fma2(d[0], f.x, ptx::fma2(ptx::pack2(r[i], r[i + 1]), kf2, e2));
        d[1] = ptx::fma2(d[1], f.y, ptx::fma2(ptx::pack2(r[i + 2], r[i + 3]), kf2, e2));
      }
    }
    ptx::tc_fence_before();
    __syncwarp();
    if (ok && lane == 0) ptx::mbar_arrive(&bars->sempty[s.slot]);
    s.next();
    // positions that a row may not see
    if (__builtin_expect((long long)(w.t + 1) * kDenseTile > w.n.min_len || pages != 3, 0)) {
      const long long t = (long long)w.t * kDenseTile + tok;
      const int* lens = reinterpret_cast<const int*>(sm + C::kLen) + buf * NR + col0;
      const bool here = pages >> (tok >> 6) & 1;
#pragma unroll
      for (int i = 0; i < HC; i += 2) {
        float2 d = ptx::unpack2(acc[i / 2]);
        if (!here || t >= lens[i]) d.x = -CUDART_INF_F;
        if (!here || t >= lens[i + 1]) d.y = -CUDART_INF_F;
        acc[i / 2] = ptx::pack2(d.x, d.y);
      }
      if (!here || t >= w.n.min_len) clean_codes<NR>(base, kslot, tok, part, here && t < w.n.max_len);
    }
    kslot = kslot + 4 >= C::kRing ? kslot + 4 - C::kRing : kslot + 4;
    // the largest operand of each row and block over the 128 positions: every warp's 32 first
    {
      float4 g = lg, top4 = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
      for (int b = 0; b < 4; ++b) {
        const uint64_t g2 = ptx::pack2(g.x, g.x);
        g = make_float4(g.y, g.z, g.w, g.x);
        float m[HC];
#pragma unroll
        for (int i = 0; i < HC / 2; ++i) {
          const float2 x = ptx::unpack2(ptx::add2(acc[i], g2));
          m[2 * i] = ptx::warp_max(x.x);
          m[2 * i + 1] = ptx::warp_max(x.y);
        }
        top4 = make_float4(top4.y, top4.z, top4.w, pick<HC>(m, lane));
      }
      if (lane < HC) ptx::sts128f(red + (quad * NR + lane) * 16, top4.x, top4.y, top4.z, top4.w);
    }
    ptx::named_bar_sync(1 + part, 128);
    float m[kRefs];                                     // this lane's blocks' largest operands
    bool stays = true;                                  // within the references' windows
    {
      float x[4][kRefs];
#pragma unroll
      for (int k = 0; k < 4; ++k) ptx::lds_floats(red + (k * NR + row) * 16 + block0 * 4, x[k]);
#pragma unroll
      for (int j = 0; j < kRefs; ++j) {
        m[j] = fmaxf(fmaxf(x[0][j], x[1][j]), fmaxf(x[2][j], x[3][j]));
        stays = stays && m[j] <= upper[j] && (m[j] > lower[j] || m[j] == -CUDART_INF_F);
      }
    }
    if constexpr (C::kReds == 2) red = red == fac ? fac + 16 * NR * 4 : fac;
    if (first || __any_sync(0xffffffffu, !stays)) {     // (the same in the part's four warps)
      // R of each block, A, and the factors by which the sums so far change when they move
      float f[kRefs], fa = 1.f, high = CUDART_NAN_F, to[kRefs];
#pragma unroll
      for (int j = 0; j < kRefs; ++j) {
        const float r = ceilf(m[j] - kTopOperand);
        // (a row without positions here, or of NaNs alone, keeps what it has)
        const bool moves = m[j] > -CUDART_INF_F && !(r <= ref[j] && r >= ref[j] - kWindow), set = ref[j] == ref[j];
        const float next = set ? fmaxf(r > ref[j] ? r + 1.f : r + kWindow / 2, top[j] - kLowest) : r + kWindow / 2;
        to[j] = moves ? next : ref[j];
        high = fmaxf(high, to[j]);
      }
#pragma unroll
      for (int o = HC; o < 32; o <<= 1) high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, o));
      if (!(level >= high - kAbove && level <= high - kAbove + kSlack)) {
        const float next = high - kAbove + kSlack / 2;
        if (level == level) fa = exp2_int((int)fminf(fmaxf(level - next, -126.f), 126.f));
        level = next;
      }
      bool moves = false;
#pragma unroll
      for (int j = 0; j < kRefs; ++j) {
        f[j] = 1.f;
        if (to[j] == to[j]) {
          const float next = fmaxf(to[j], level - kFactor);
          if (ref[j] == ref[j]) f[j] = exp2_int((int)fminf(fmaxf(ref[j] - next, -126.f), 126.f));
          top[j] = ref[j] == ref[j] ? fmaxf(top[j], next) : next;
          ref[j] = next;
          upper[j] = next + kTopOperand;                // (one that is as low as it may be stays below its window)
          lower[j] = next <= fmaxf(top[j] - kLowest, level - kFactor) ? -CUDART_INF_F : upper[j] - 1.f - kWindow;
        }
        moves |= f[j] != 1.f;
      }
      const bool moved = __any_sync(0xffffffffu, moves);
      if (__any_sync(0xffffffffu, fa != 1.f)) {
        if (lane < HC) ptx::sts32f(row_na + lane * 4, fa);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < HC / 2; i += 2) {
          const ulonglong2 by = ptx::lds128_pairs(row_na + i * 8);
          l[i] = ptx::mul2(l[i], by.x);
          l[i + 1] = ptx::mul2(l[i + 1], by.y);
        }
        __syncwarp();
      }
      if (moved) {
        wait_pv();
#pragma unroll 1
        for (int b = 0; b < 4; ++b) {
          float fb = f[0];                                // of block b, in the lanes that keep its reference
#pragma unroll
          for (int j = 1; j < kRefs; ++j) fb = block0 + j == b ? f[j] : fb;
          const bool mine = block0 <= b && b < block0 + kRefs;
          uint32_t rows = __ballot_sync(0xffffffffu, mine && fb != 1.f);
          if (rows == 0) continue;
          if constexpr (HC < 32) rows = rows >> (b / kRefs * HC) & ((1u << HC) - 1u);
          if (mine) ptx::sts32f(row_na + row * 4, fb);
          __syncwarp();
          const uint32_t at = lane_base + C::kOCols * b + col0;
#pragma unroll 1
          for (int i0 = 0; i0 < HC; i0 += kChunk) {
            if (!(rows >> i0 & 0xffu)) continue;
            const float4 f0 = ptx::lds128f(row_na + i0 * 4), f1 = ptx::lds128f(row_na + i0 * 4 + 16);
            const float by[kChunk] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
            uint32_t x[C::kPasses == 1 ? 2 : 1][kChunk];
            tmem_ld<kChunk>(at + i0, x[0]);
            if constexpr (C::kPasses == 1) tmem_ld<kChunk>(at + NR + i0, x[1]);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < kChunk; ++i) {
              x[0][i] = __float_as_uint(__uint_as_float(x[0][i]) * by[i]);
              if constexpr (C::kPasses == 1) x[1][i] = __float_as_uint(__uint_as_float(x[1][i]) * by[i]);
            }
            tmem_st<kChunk>(at + i0, x[0]);
            if constexpr (C::kPasses == 1) tmem_st<kChunk>(at + NR + i0, x[1]);
          }
          __syncwarp();
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
      }
      if (lane < HC) ptx::sts32f(row_na + lane * 4, level == level ? -level : 0.f);
#pragma unroll
      for (int j = 0; j < kRefs; ++j) {
        const int k = (int)fminf(fmaxf(level - ref[j], -14.f), kFactor);
        ptx::sts16(row_c + ((block0 + j) * HC + row) * 2, ref[j] == ref[j] ? (uint16_t)((15 + k) << 10) : 0);   // 2^k
      }
      __syncwarp();
    }
    // weights
    const float down = exp2_int(-e);
    uint32_t w16[HC / 2];
    {
      const uint64_t down2 = ptx::pack2(down, down);
#pragma unroll
      for (int i = 0; i < HC / 2; i += 2) {
        const ulonglong2 na = ptx::lds128_pairs(row_na + i * 8);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 x = ptx::unpack2(ptx::add2(acc[i + j], j ? na.y : na.x));
          const float a = ptx::ex2_approx(x.x), b = ptx::ex2_approx(x.y);
          l[i + j] = ptx::fma2(ptx::pack2(a, b), down2, l[i + j]);
          w16[i + j] = as_u32(__floats2half2_rn(a, b));
        }
      }
    }
    // block b's operand: w m_b 2^(A - R_b) as hi + lo.  The offset: odd multiples of 2^-7 half steps, one per position
    {
      float4 rot = v4;
      const __half2 up = __float2half2_rn(C::kLoUp);
      const __half2 dither = __float2half2_rn((float)(2 * (int)(__brev(tok) >> 25) - 127) * (0x1p-17f / C::kLoUp));
#pragma unroll 1
      for (int b = 0; b < 4; ++b) {
        const __half2 m = __float2half2_rn(rot.x * down);
        rot = make_float4(rot.y, rot.z, rot.w, rot.x);
        uint32_t hi[HC / 4], lo[HC / 4];
#pragma unroll
        for (int i = 0; i < HC / 4; i += 2) {
          const uint4 c8 = ptx::lds128(row_c + (b * HC + 4 * i) * 2);
          const uint32_t cs[4] = {c8.x, c8.y, c8.z, c8.w};
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const __half2 x = __hfma2(__hmul2(as_half2(w16[2 * (i + j)]), m), as_half2(cs[2 * j]), dither);
            const __half2 y = __hfma2(__hmul2(as_half2(w16[2 * (i + j) + 1]), m), as_half2(cs[2 * j + 1]), dither);
            hi[i + j] = f16x4_to_e4m3x4(as_u32(x), as_u32(y));
            uint32_t bx, by;
            e4m3x4_to_f16x4(hi[i + j], bx, by);
            __half2 dx = __hsub2(x, as_half2(bx)), dy = __hsub2(y, as_half2(by));
            if constexpr (C::kPasses == 1) {
              dx = __hmul2(dx, up);
              dy = __hmul2(dy, up);
            }
            lo[i + j] = f16x4_to_e4m3x4(as_u32(dx), as_u32(dy));
          }
        }
        SMLA_WAIT(&bars->pempty[pb.slot], pb.parity ^ 1);
        const uint32_t dst = base + C::kP + pb.slot * C::kPBuf;
        if constexpr (HC >= 16) {
#pragma unroll
          for (int u = 0; u < HC / 16; ++u) {
            ptx::sts128_async_only(dst + swz_row<C::kPRow>(tok, col0 / 16 + u),
                                   make_uint4(hi[4 * u], hi[4 * u + 1], hi[4 * u + 2], hi[4 * u + 3]));
            ptx::sts128_async_only(dst + swz_row<C::kPRow>(tok, (NR + col0) / 16 + u),
                                   make_uint4(lo[4 * u], lo[4 * u + 1], lo[4 * u + 2], lo[4 * u + 3]));
          }
        } else {
          ptx::sts64_async_only(dst + swz_row<C::kPRow>(tok, 0) + col0, hi[0], hi[1]);
          ptx::sts64_async_only(dst + swz_row<C::kPRow>(tok, 1) + col0, lo[0], lo[1]);
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (ok && lane == 0) ptx::mbar_arrive(&bars->pfull[pb.slot]);
        if (b == 3) last_par = pb.parity;
        pb.next();
      }
    }

    const bool last = w.last_of_segment(), ends = w.t == w.n.tiles - 1;
    whole = begins && ends;
    w.next();
    first = last;
  }
}

// ----------------------------------------------------------------------------- kernel

// The line that is shared out: each item is kStart units and then its tiles.  A CTA that goes on to a further item spends
// about two tiles' time on it (the item's rows read, the last one's results written, the pipeline filled again), so its
// run is shorter by as much; while not every CTA has a tile, nothing is set aside.  Measured, when tiles took less (1.9, 2.5
// and 3.6 us for 16, 32 and 64 rows), with tiles alone / with starts of 1 / 2 / 3 tiles: 18 requests x 8192 positions of 64
// heads 64.1 / 60.2 / 57.2 / 57.4 us, 96 ragged requests of 16 heads 80.5 / 77.0 / 73.8 / 73.7, 40 x 8192 of 32 heads 63.0 /
// 60.8 / 59.3 / 59.5.
constexpr int kStart = 2;

// This CTA's run: the units [a, e) of the line, for T tiles and n items.
__device__ __forceinline__ void run_bounds(const DenseParams& p, long long T, int n, Bars* bars, bool write, int& start,
                                           long long& a, long long& e) {
  start = T >= p.ctas ? kStart : 0;
  const long long units = T + (long long)start * n;
  const int active = (int)min((long long)p.ctas, units), c = blockIdx.x;
  a = c < active ? run_start(units, active, c) : units;
  e = c < active ? run_start(units, active, c + 1) : units;
  if (write) {
    bars->units = units;
    bars->active = active;
  }
}

// The items in which the run begins and ends, if they are among i0 .. i1 - 1, whose `mine` tiles begin at tile `at`.
__device__ __forceinline__ void find_ends(const DenseParams& p, Bars* bars, int i0, int i1, long long at, long long mine,
                                          int start, long long a, long long e) {
  if (a >= e || a >= at + mine + (long long)start * i1 || e <= at + (long long)start * i0) return;
  long long x = at;
#pragma unroll 1
  for (int i = i0; i < i1; ++i) {
    const int tiles = lens_of(p, rows_of(p, i)).tiles;
    const long long begin = x + (long long)start * (i + 1), end = begin + tiles;       // the item's tiles on the line
    const long long from = max(a, begin), to = min(e, end);
    if (from < to) {
      if (a >= begin - start) {                          // nothing of the items before
        bars->first_item = i;
        bars->first_tile = (int)(from - begin);
        bars->run_begin = x + (from - begin);
      }
      if (e <= end + start) {                            // nor of those behind
        bars->last_item = i;
        bars->last_begin = begin;
        bars->last_end = end;
        bars->run_end = x + (to - begin);
      }
    }
    x += tiles;
  }
}

// A table of at most two pages gives every item one tile: no lengths to add up, nothing to merge (1 x 77 positions 9.2 us
// instead of 10.2).
__host__ __device__ __forceinline__ bool one_tile(const DenseParams& p) { return p.max_pages <= 2; }

// Every CTA adds up the tiles of all items.  Few items: one warp, up to four items per lane (the general search's code
// and barriers take 0.7 us more of a call: 1 x 77 positions 11.0 us instead of 10.3).  Else a run of items per thread,
// then a scan of the threads' sums.
template <int kThreads>
__device__ __forceinline__ void find_run(const DenseParams& p, unsigned char* scratch, Bars* bars) {
  if (one_tile(p)) {                                     // an item is a tile: nothing to look up
    if (threadIdx.x == 0) {
      const int n = p.requests * p.groups, active = min(p.ctas, n), c = min((int)blockIdx.x, active);
      bars->units = n;
      bars->active = active;
      bars->run_begin = run_start(n, active, c);
      bars->run_end = c < active ? run_start(n, active, c + 1) : n;
      bars->first_item = (int)bars->run_begin;
      bars->first_tile = 0;
      bars->last_item = (int)bars->run_end - 1;
      bars->last_begin = bars->run_end - 1;
      bars->last_end = bars->run_end;
    }
    __syncthreads();
    return;
  }
  if (threadIdx.x == 0) bars->run_begin = bars->run_end = 0;
  if (p.requests * p.groups <= 128) {
    if (threadIdx.x < 32) {
      const int n = p.requests * p.groups, per = (n + 31) >> 5, lane = threadIdx.x;
      const int i0 = min(n, lane * per), i1 = min(n, i0 + per);
      long long mine = 0;
#pragma unroll 1
      for (int i = i0; i < i1; ++i) mine += lens_of(p, rows_of(p, i)).tiles;
      __syncwarp();                                      // the empty run is written
      long long upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += up;
      }
      long long a, e;
      int start;
      run_bounds(p, __shfl_sync(0xffffffffu, upto, 31), n, bars, lane == 0, start, a, e);
      find_ends(p, bars, i0, i1, upto - mine, mine, start, a, e);
    }
    __syncthreads();
    return;
  }
  constexpr int kPer = kThreads / 32;
  long long* sums = reinterpret_cast<long long*>(scratch);
  const int n = p.requests * p.groups, per = (n + kThreads - 1) / kThreads;
  const int i0 = min(n, (int)threadIdx.x * per), i1 = min(n, i0 + per);
  long long mine = 0;
#pragma unroll 1
  for (int i = i0; i < i1; ++i) mine += lens_of(p, rows_of(p, i)).tiles;
  sums[threadIdx.x] = mine;
  __syncthreads();
  if (threadIdx.x < 32) {                                // exclusive prefix over kPer sums per lane
    long long v[kPer], part = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      v[j] = part;
      part += sums[kPer * threadIdx.x + j];
    }
    long long before = part;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, before, o);
      if ((int)threadIdx.x >= o) before += up;
    }
    if (threadIdx.x == 31) bars->units = before;
    before -= part;
#pragma unroll
    for (int j = 0; j < kPer; ++j) sums[kPer * threadIdx.x + j] = before + v[j];
  }
  __syncthreads();
  long long a, e;
  int start;
  const long long T = bars->units;
  __syncthreads();
  run_bounds(p, T, n, bars, threadIdx.x == 0, start, a, e);
  find_ends(p, bars, i0, i1, sums[threadIdx.x], mine, start, a, e);
  __syncthreads();
}

__device__ __forceinline__ RunDesc describe_run(const Bars* bars) {
  const int c = blockIdx.x, active = bars->active;
  const long long T = bars->units, end = bars->last_end;
  if (bars->run_begin == bars->run_end || bars->last_begin < run_start(T, active, c) || end <= run_start(T, active, c + 1))
    return RunDesc{0, 0};
  int c1 = (int)((end * active + T - 1) / T);            // first CTA past the item, give or take one
  while (c1 > c && run_start(T, active, c1) >= end) --c1;
  while (c1 + 1 < active && run_start(T, active, c1 + 1) < end) ++c1;
  return RunDesc{bars->last_item, c1 - c + 1};
}

template <int NR>
__global__ void __launch_bounds__(DC<NR>::kThreads, 1)
    dense_kernel(const DenseParams p, const __grid_constant__ CUtensorMap map, const __grid_constant__ CUtensorMap smap,
                 RunDesc* descs, float* lse_part, float* o_part) {
  using C = DC<NR>;
  extern __shared__ __align__(1024) unsigned char sm[];
  const uint32_t base = ptx::smem_u32(sm);
  Bars* bars = reinterpret_cast<Bars*>(sm + C::kBar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) ptx::griddep_launch_dependents();   // the merge, which waits for this grid's results
  const int role = warp - C::kSoftWarps;                 // of the warps behind the softmax warps
  if (role == kCopyRole) init_bars<C::kSoftWarps>(bars, p, lane, &map, &smap);
  if (role == kQkRole) {
    ptx::tmem_alloc(&bars->tmem, C::kTmemCols);
    ptx::tmem_relinquish();
  }
  find_run<C::kThreads>(p, sm, bars);            // the scratch is overwritten by the pipeline afterwards
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = bars->tmem;

  if (role < 0) {
    ptx::setmaxnreg_inc<C::kSoftRegs>();
    softmax_role<NR>(p, sm, base, tmem, bars, warp, lane, o_part, lse_part);
  } else {
    ptx::setmaxnreg_dec<C::kMiscRegs>();
    if (role == kCopyRole) copy_role<NR>(p, &map, &smap, base, bars, lane);
    else if (role == kQkRole) qk_role<NR>(p, base, tmem, bars, lane);
    else if (role == kPvRole) pv_role<NR>(p, base, tmem, bars, lane);
    else if (lane == 0) descs[blockIdx.x] = describe_run(bars);
  }

  // nothing of this CTA's may be in flight when it leaves: the MMAs (their last commits) and, after a wait
  // that gave up, the copies
  __syncthreads();
  int never = 0;
  if (role == kCopyRole && bars->abort) {
    drain_copies(bars->kfull, bars->armed_k, C::kRing, lane);
    drain_copies(bars->rfull, bars->armed_r, C::kRopeSlots, lane);
    drain_copies(bars->scfull, bars->armed_sc, C::kScaleSlots, lane);
  }
  if (role == kQkRole) {
    ptx::mbar_wait_warp(&bars->drain[0], 0, &never, lane, 100000000ull);
    ptx::mbar_wait_warp(&bars->drain[1], 0, &never, lane, 100000000ull);
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::kTmemCols);
  }
  if (threadIdx.x == 0 && bars->abort) atomicOr(p.err, SMLA_DEVERR_TIMEOUT);
}

// ----------------------------------------------------------------------------- merge

constexpr int kMergeThreads = 128;
constexpr int kMergeBatch = 8;            // partial rows in flight per thread
constexpr int kFewParts = 16;             // items of at most so many parts: one warp per (row, 128 dims)

// The partials of one row: part 0 in slot 1 of CTA c, part s in slot 0 of CTA c + s.
struct PartRows {
  int c, row, nr;
  __device__ __forceinline__ size_t at(int s) const { return (s == 0 ? 2 * (size_t)c + 1 : 2 * (size_t)(c + s)) * nr + row; }
};

__device__ __forceinline__ void add_part(float4& acc, float w, const float4& v) {
  acc.x = fmaf(w, v.x, acc.x);
  acc.y = fmaf(w, v.y, acc.y);
  acc.z = fmaf(w, v.z, acc.z);
  acc.w = fmaf(w, v.w, acc.w);
}

__device__ __forceinline__ void store_joined(const DenseParams& p, size_t row, int block, int lane, const float4& v,
                                             float lse) {
  reinterpret_cast<uint2*>(p.out + row * kDLatent + 128 * block)[lane] =
      make_uint2(f32x2_to_bf16x2(v.x, v.y), f32x2_to_bf16x2(v.z, v.w));
  if (lane == 0 && block == 0) p.lse[row] = lse;
}

// Joins the partials of the items that cross CTA runs: lse = ln sum_s exp(lse_s), out = sum_s exp(lse_s - lse)
// o_s.  An item that begins in CTA c and ends in CTA c1 left its partials in slot 1 of c and slot 0 of
// c + 1 .. c1.  Every CTA lists those items from the run descriptors, in the same order, and takes its share of their
// (row, 128 dims).  Bound by the latency of the partials (in L2): an item of few parts, of which a batch has many,
// takes one warp, all its loads in flight at once and no barrier; in one of many parts (a single long request) four
// warps share the parts.  Measured, whole calls with four warps / one warp (the decode itself took less then): 32 x 2048
// positions of 64 heads (6 parts) 62 / 50 us, 10 x 8192 of 64 heads (16 parts) 42.3 / 38.5 us, 10 x 8192 of 16 heads 23.1 /
// 24.8 us; of 64 parts and more one warp would take its loads in eight rounds.
// This grid is resident while the decode's still writes, so partials are read from L2, not through the read-only path.
__global__ void __launch_bounds__(kMergeThreads) dense_merge_kernel(const DenseParams p, const RunDesc* descs,
                                                                    const float* lse_part, const float* o_part) {
  __shared__ int parts_s[kDenseMaxCtas], item_s[kDenseMaxCtas];     // of the item that begins in CTA c, 0: none to join
  __shared__ uint16_t order_s[kDenseMaxCtas];                       // few parts from the front, many from the back
  __shared__ float w_s[kDenseMaxCtas];
  __shared__ int few_s, many_s;
  __shared__ float lse_s;
  __shared__ float4 sum_s[4][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  ptx::griddep_wait();
  for (int c = tid; c < p.ctas; c += kMergeThreads) {
    const RunDesc d = descs[c];
    parts_s[c] = d.parts;
    item_s[c] = d.item;
  }
  __syncthreads();
  if (warp == 0) {
    int few = 0, many = 0;
    const uint32_t below = (1u << lane) - 1;
    for (int c0 = 0; c0 < p.ctas; c0 += 32) {
      const int parts = c0 + lane < p.ctas ? parts_s[c0 + lane] : 0;
      const uint32_t f = __ballot_sync(0xffffffffu, parts > 0 && parts <= kFewParts);
      const uint32_t m = __ballot_sync(0xffffffffu, parts > kFewParts);
      if (f >> lane & 1) order_s[few + __popc(f & below)] = (uint16_t)(c0 + lane);
      if (m >> lane & 1) order_s[kDenseMaxCtas - 1 - many - __popc(m & below)] = (uint16_t)(c0 + lane);
      few += __popc(f);
      many += __popc(m);
    }
    if (lane == 0) {
      few_s = few;
      many_s = many;
    }
  }
  __syncthreads();
  const int nr = p.nr;
  for (int idx = blockIdx.x * (kMergeThreads / 32) + warp; idx < few_s * nr * 4; idx += gridDim.x * (kMergeThreads / 32)) {
    const int c = order_s[idx / (4 * nr)], row = (idx >> 2) % nr, block = idx & 3, parts = parts_s[c];
    const Rows it = rows_of(p, item_s[c]);
    if (row >= it.nrows) continue;
    const PartRows rows{c, row, nr};
    const float4* o = reinterpret_cast<const float4*>(o_part) + 32 * block + lane;
    const float x = lane < parts ? __ldcg(lse_part + rows.at(lane)) : -CUDART_INF_F;
    float4 v[kMergeBatch];
#pragma unroll
    for (int s = 0; s < kMergeBatch; ++s)
      if (s < parts) v[s] = __ldcg(o + rows.at(s) * (kDLatent / 4));
    float m = x;
#pragma unroll
    for (int h = 16; h; h >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, h));
    if (__any_sync(0xffffffffu, isnan(x))) m = CUDART_NAN_F;
    const float e = m == -CUDART_INF_F ? 0.f : expf(x - m);
    float z = e;
#pragma unroll
    for (int h = 16; h; h >>= 1) z += __shfl_xor_sync(0xffffffffu, z, h);
    const float w = z == 0.f ? 0.f : e / z;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int s = 0; s < kMergeBatch; ++s)
      if (s < parts) add_part(acc, __shfl_sync(0xffffffffu, w, s), v[s]);
#pragma unroll
    for (int s = kMergeBatch; s < kFewParts; ++s)
      if (s < parts) v[s - kMergeBatch] = __ldcg(o + rows.at(s) * (kDLatent / 4));
#pragma unroll
    for (int s = kMergeBatch; s < kFewParts; ++s)
      if (s < parts) add_part(acc, __shfl_sync(0xffffffffu, w, s), v[s - kMergeBatch]);
    store_joined(p, (size_t)it.req * p.q_per_req * p.H + it.row0 + row, block, lane, acc,
                 z == 0.f ? -CUDART_INF_F : m + logf(z));
  }
  for (int idx = blockIdx.x; idx < many_s * nr * 4; idx += gridDim.x) {
    const int c = order_s[kDenseMaxCtas - 1 - idx / (4 * nr)], row = (idx >> 2) % nr, block = idx & 3, parts = parts_s[c];
    const Rows it = rows_of(p, item_s[c]);
    if (row >= it.nrows) continue;                       // uniform over the CTA
    // warp w takes parts w, w + 4, ...: their rows in flight before the weights are known
    const PartRows rows{c, row, nr};
    const float4* o = reinterpret_cast<const float4*>(o_part) + 32 * block + lane;
    float4 v[kMergeBatch];
#pragma unroll
    for (int s = 0; s < kMergeBatch; ++s)
      if (warp + 4 * s < parts) v[s] = __ldcg(o + rows.at(warp + 4 * s) * (kDLatent / 4));
    __syncthreads();                                     // w_s and sum_s of the row before have been read
    if (warp == 0) {
      float m = -CUDART_INF_F;
      bool bad = false;
      for (int s = lane; s < parts; s += 32) {
        const float x = __ldcg(lse_part + rows.at(s));
        bad |= isnan(x);
        m = fmaxf(m, x);
        w_s[s] = x;
      }
#pragma unroll
      for (int h = 16; h; h >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, h));
      if (__any_sync(0xffffffffu, bad)) m = CUDART_NAN_F;
      float z = 0.f;
      for (int s = lane; s < parts; s += 32) {
        const float e = m == -CUDART_INF_F ? 0.f : expf(w_s[s] - m);
        w_s[s] = e;
        z += e;
      }
#pragma unroll
      for (int h = 16; h; h >>= 1) z += __shfl_xor_sync(0xffffffffu, z, h);
      const float inv = z == 0.f ? 0.f : 1.f / z;
      for (int s = lane; s < parts; s += 32) w_s[s] *= inv;
      if (lane == 0) lse_s = z == 0.f ? -CUDART_INF_F : m + logf(z);
    }
    __syncthreads();
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; warp + 4 * s0 < parts; s0 += kMergeBatch) {
      if (s0 > 0) {
#pragma unroll
        for (int s = 0; s < kMergeBatch; ++s)
          if (warp + 4 * (s0 + s) < parts) v[s] = __ldcg(o + rows.at(warp + 4 * (s0 + s)) * (kDLatent / 4));
      }
#pragma unroll
      for (int s = 0; s < kMergeBatch; ++s)
        if (warp + 4 * (s0 + s) < parts) add_part(acc, w_s[warp + 4 * (s0 + s)], v[s]);
    }
    sum_s[warp][lane] = acc;
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int s = 1; s < 4; ++s) add_part(acc, 1.f, sum_s[s][lane]);
      store_joined(p, (size_t)it.req * p.q_per_req * p.H + it.row0 + row, block, lane, acc, lse_s);
    }
  }
}

// ----------------------------------------------------------------------------- host

// Workspace: header (error word), run descriptors, lse partials [2 ctas][NR], row partials [2 ctas][NR][512].
constexpr size_t kDescBytes = (kDenseMaxCtas * sizeof(RunDesc) + 255) / 256 * 256;
size_t lse_part_bytes(int ctas, int nr) { return ((size_t)2 * ctas * nr * sizeof(float) + 255) / 256 * 256; }

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encoder() {
  static const EncodeTiled fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeTiled>(f);
  }();
  return fn;
}

// The cache as [page][record][byte], in boxes of 64 records of one page, `bytes` wide.
bool encode_map(CUtensorMap* map, const DenseParams& p, uint32_t bytes, CUtensorMapSwizzle swizzle) {
  const cuuint64_t dims[3] = {kRecordBytes, kPageSize, (cuuint64_t)p.num_pages};
  const cuuint64_t strides[2] = {kRecordBytes, (cuuint64_t)kRecordBytes * kPageSize};
  const cuuint32_t box[3] = {bytes, kPageSize, 1}, step[3] = {1, 1, 1};
  return encoder()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(p.kv), dims, strides, box, step,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NR>
cudaError_t launch_nr(const DenseParams& p, unsigned char* ws, cudaStream_t stream) {
  CUtensorMap map, smap;
  if (!encoder() || !encode_map(&map, p, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_map(&smap, p, 16, CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorNotSupported;
  // the shared-memory attribute belongs to the device's copy of the kernel: set once per device
  static std::atomic<bool> set[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !set[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(dense_kernel<NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, DC<NR>::kBytes);
    if (e != cudaSuccess) return e;
    if (dev < 64) set[dev].store(true, std::memory_order_relaxed);
  }
  RunDesc* descs = reinterpret_cast<RunDesc*>(ws + kWorkspaceHeader);
  float* lse_part = reinterpret_cast<float*>(ws + kWorkspaceHeader + kDescBytes);
  float* o_part = reinterpret_cast<float*>(ws + kWorkspaceHeader + kDescBytes + lse_part_bytes(p.ctas, NR));
  dense_kernel<NR><<<p.ctas, DC<NR>::kThreads, DC<NR>::kBytes, stream>>>(p, map, smap, descs, lse_part, o_part);
  e = cudaGetLastError();
  if (e != cudaSuccess || one_tile(p)) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(8 * p.ctas);
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = stream;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = a;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, dense_merge_kernel, p, (const RunDesc*)descs, (const float*)lse_part,
                            (const float*)o_part);
}

}  // namespace

cudaError_t launch_dense(const DenseParams& p, cudaStream_t stream) {
  unsigned char* ws = reinterpret_cast<unsigned char*>(p.err);    // the workspace begins with the error word
  if (p.nr == 16) return launch_nr<16>(p, ws, stream);
  if (p.nr == 32) return launch_nr<32>(p, ws, stream);
  return launch_nr<64>(p, ws, stream);
}

}  // namespace smla

using namespace smla;

extern "C" int sparse_mla_dense_plan_for(const smla_dense_dims* d, int32_t sm_count, smla_dense_plan* plan) {
  if (!d || !plan || sm_count < 1) return SMLA_ERR_INVALID_ARG;
  if (d->batch < 1 || d->num_heads < 1 || d->max_pages_per_seq < 1 || d->num_pages < 1 || d->ctas < 0 ||
      d->queries_per_request < 0)
    return SMLA_ERR_INVALID_ARG;
  const int sq = d->queries_per_request > 1 ? d->queries_per_request : 1;
  if (d->batch % sq != 0) return SMLA_ERR_INVALID_ARG;
  if (d->page_size != kPageSize || d->d_latent != kDLatent || d->d_rope != kDRope) return SMLA_ERR_UNSUPPORTED;
  if (d->batch > kMaxBatch || d->num_heads > kDenseMaxHeads || d->num_pages > 0x7fffffff || d->ctas > kDenseMaxCtas)
    return SMLA_ERR_UNSUPPORTED;
  const int64_t rows = (int64_t)sq * d->num_heads;
  plan->ctas = d->ctas > 0 ? d->ctas : (sm_count < kDenseMaxCtas ? sm_count : kDenseMaxCtas);
  plan->reserved = 0;
  // Rows that a CTA takes through a tile together.  Few rows: a tile is done sooner (1.9, 2.8 and 4.2 us for 16, 32
  // and 64 rows), and so are the steps around the tiles (a CTA's rows read and its results written), but each row
  // group reads the tile again.  Measured at 64 heads, 16 / 32 / 64 rows: 1 request x 8192 positions 19.2 / 19.4 / 23.8
  // us, 4 x 8192 28.5 / 26.9 / 31.5, 32 x 4096 80.0 / 60.7 / 60.9, 32 x 8192 133 / 94 / 86, 32 x 16384 235 / 157 / 136.  So:
  // the fewest rows with which a CTA has at most a few tiles if every request is as long as its table.
  const int64_t tiles = d->batch / sq * ((d->max_pages_per_seq + (int64_t)1) / 2);
  auto groups = [&](int nr) { return (rows + nr - 1) / nr; };
  if (rows <= 16 || tiles * groups(16) <= kMostTiles16 * (int64_t)plan->ctas) plan->rows_per_cta = 16;
  else if (rows <= 32 || tiles * groups(32) <= kMostTiles32 * (int64_t)plan->ctas) plan->rows_per_cta = 32;
  else plan->rows_per_cta = 64;
  plan->row_groups = (int32_t)groups(plan->rows_per_cta);
  // a CTA counts its tiles in 32 bits
  const int64_t most = tiles * plan->row_groups;
  if (most / plan->ctas >= 0x7fffffff) return SMLA_ERR_UNSUPPORTED;
  plan->workspace_bytes = kWorkspaceHeader + kDescBytes + lse_part_bytes(plan->ctas, plan->rows_per_cta) +
                          (size_t)2 * plan->ctas * plan->rows_per_cta * kDLatent * sizeof(float);
  return SMLA_OK;
}
