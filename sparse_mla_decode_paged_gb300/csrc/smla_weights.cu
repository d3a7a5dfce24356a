// Attention weights accumulated per cached position:
//
//   w[r][t] = decay w[r][t] + sum over the request's queries b and heads h of exp(sm_scale q[b][h].k_t - lse[b][h]),
//
// t below seq_lens[b]; rows with an lse of -inf saw nothing and add nothing.  The codes go to the tensor core as they are, q as
// two E4M3 terms that are exact but for elements below 2^-9 of the row's largest, the scales and the sums stay in fp32 (as the
// dense decode's scores; no values are read).
// S^T of a tile: M = 128 positions, N = the rows, one accumulator per 128-dim scale block and one for the rope, so a thread
// has one position and half of the rows: it forms their scores and adds up the weights in registers; no maximum is needed, lse
// is given.  The two halves of a position meet in shared memory, always in the same order.
//
// Tiles of 128 positions, laid end to end over the requests, are shared out in equal runs.  Up to 128 rows of q stay in shared
// memory over a run; more rows go through the tiles in groups, kSub tiles at a time so that the records are found in L2 again.
// What bounds it: HBM bytes (656 per position) for up to 128 rows.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <atomic>
#include <cstddef>

#include "smla_dense_parts.cuh"
#include "smla_device.cuh"
#include "smla_internal.h"
#include "smla_ptx.cuh"
#include "smla_split_layout.cuh"

namespace smla {
namespace {

constexpr uint32_t kSlot = 16384;         // 128 positions x 128 bytes: one code block or the rope of a tile
constexpr int kChunks = 5;                // of a tile: the four code blocks, then the rope
constexpr int kSoftWarps = 8;             // warp w: TMEM lanes of quadrant w % 4, row half w / 4
constexpr int kThreads = 32 * (kSoftWarps + 2);
constexpr int kCopyWarp = kSoftWarps, kMmaWarp = kSoftWarps + 1;
constexpr int kSub = 8;
// Tiles between a tile's prefetch into L2 and its copy (32 x 32768 positions of 16, 32, 64 heads: 111, 115, 134 us, none 121,
// 122, 133, two 118 and 141 for 16 and 64).
constexpr int kAhead = 1;
constexpr uint64_t kLeastWaitNs = 1000;   // limits below this are meant to run out: nothing is issued

template <int NR>
struct WC {
  // hi and lo terms of q: one MMA of twice the columns up to 64 rows, which meet in registers, else two MMAs (64 rows: 124 us
  // for 32 x 32768 positions, 134 with two MMAs, which read the codes twice)
  static constexpr int kPasses = NR >= 128 ? 2 : 1;
  static constexpr int kCols = NR >= 128 ? NR : 2 * NR;               // columns of a score accumulator
  static constexpr int kSBufs = NR >= 64 ? 4 : 5;
  static constexpr uint32_t kTmemCols = NR >= 64 ? 512 : NR == 32 ? 512 : 256;
  static constexpr int kRing = NR == 128 ? 4 : NR == 64 ? 8 : 10;    // slots of code blocks and ropes
  static constexpr int kScaleSlots = 3;
  static constexpr int HC = NR / 2;                                  // rows of a softmax thread
  static constexpr uint32_t kQ8Chunk = 2 * NR * 128;
  static constexpr uint32_t kQr = 4 * kQ8Chunk;
  static constexpr uint32_t kK = (kQr + NR * 128 + 1023) / 1024 * 1024;
  static constexpr uint32_t kScale = kK + kRing * kSlot;
  static constexpr uint32_t kRows = kScale + kScaleSlots * 2048;     // [2][3][NR]: factor, -lse log2 e, length
  static constexpr uint32_t kSum = kRows + 2 * 3 * NR * 4;           // [2][128] float
  static constexpr uint32_t kBar = kSum + 2 * 128 * 4;
  static constexpr uint32_t kBytes = kBar + 512;
  static_assert(kBytes <= 232448, "shared memory");
  static_assert(kSBufs * kCols <= (int)kTmemCols, "TMEM");
};

struct Bars {
  uint64_t kfull[10], kempty[10], sfull[5], sempty[5], scfull[3], scempty[3], qfull, drain;
  uint32_t tmem;
  int abort;
  int armed_k[10], armed_sc[3];
  int pages_ok[3];                        // of the tile in each scale slot: bit h: page h is loaded
  int first_req, first_tile, run;         // this CTA's run of tiles
  long long sums[kThreads / 32];
};
static_assert(sizeof(Bars) <= 512, "barrier area");

__device__ __forceinline__ int clamped_len(const WeightsParams& p, int b) {
  const long long most = min((long long)p.max_pages * kPageSize, (long long)p.cols);
  return (int)min((long long)max(__ldg(p.seq_lens + b), 0), most);
}

// The longest of a request's queries.
__device__ __forceinline__ int longest(const WeightsParams& p, int req) {
  int n = 0;
#pragma unroll 1
  for (int b = req * p.q_per_req; b < (req + 1) * p.q_per_req; ++b) n = max(n, clamped_len(p, b));
  return n;
}

__device__ __forceinline__ int tiles_of(int len) { return (int)(((long long)len + kDenseTile - 1) / kDenseTile); }

// Walks (request, tile, row group) of a run: kSub tiles of a request with each group in turn.
struct Walk {
  int req, t, left, len = 0, tiles = 0, group = 0, from, to = 0;
  bool entered = false;
  __device__ __forceinline__ explicit Walk(const Bars* bars) : req(bars->first_req), t(bars->first_tile), left(bars->run) {}
  __device__ __forceinline__ bool here(const WeightsParams& p) {
#pragma unroll 1
    while (left > 0 && !entered) {
      len = longest(p, req);
      tiles = tiles_of(len);
      if (tiles == 0) {
        ++req;
        continue;
      }
      entered = true;
      begin(p);
    }
    return left > 0;
  }
  __device__ __forceinline__ void begin(const WeightsParams& p) {
    from = t;
    to = min(tiles, t + left);
    if (p.groups > 1) to = min(to, t + kSub);
  }
  __device__ __forceinline__ void next(const WeightsParams& p) {
    if (++t < to) return;
    if (++group < p.groups) {
      t = from;
      return;
    }
    group = 0;
    left -= to - from;
    if (t == tiles) {
      t = 0;
      ++req;
      entered = false;
    } else if (left > 0) {
      begin(p);
    }
  }
};

__device__ __forceinline__ int page_entry(const WeightsParams& p, int req, int len, int lp) {
  return (long long)lp * kPageSize < len ? __ldg(p.block_table + (size_t)req * p.max_pages + lp) : -1;
}

template <int NR>
__device__ void copy_role(const WeightsParams& p, const CUtensorMap* map, const CUtensorMap* smap, uint32_t base,
                          Bars* bars, int lane) {
  using C = WC<NR>;
  Walk w(bars);
  Ring<C::kRing> k;
  Ring<C::kScaleSlots> sc;
  uint32_t ok = p.wait_ns >= kLeastWaitNs;
  int cur = 0, nxt = 0, base_lp = 0, req = -1, next_lp = -1;     // block-table entries of 16 tiles, one lane each
#pragma unroll 1
  while (w.here(p)) {
    const int lp = 2 * w.t;
    if (req != w.req || lp != next_lp) {
      if (req != w.req && w.group == 0 && lane == 0 && p.err)
        for (int b = w.req * p.q_per_req; b < (w.req + 1) * p.q_per_req; ++b)
          if (__ldg(p.seq_lens + b) > clamped_len(p, b)) atomicOr(p.err, SMLA_DEVERR_LEN_RANGE);
      req = w.req;
      base_lp = lp;
      cur = page_entry(p, req, w.len, lp + lane);
      nxt = page_entry(p, req, w.len, lp + 32 + lane);
    } else if (lp == base_lp + 32) {
      base_lp = lp;
      cur = nxt;
      nxt = page_entry(p, req, w.len, lp + 32 + lane);
    }
    next_lp = lp + 2;
    const int pg[2] = {__shfl_sync(0xffffffffu, cur, lp - base_lp), __shfl_sync(0xffffffffu, cur, lp - base_lp + 1)};
    int good = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool used = (long long)(lp + h) * kPageSize < w.len;
      const bool in_cache = pg[h] >= 0 && (int64_t)pg[h] < p.num_pages;
      if (used && in_cache) good |= 1 << h;
      if (used && !in_cache && lane == 0 && p.err) atomicOr(p.err, SMLA_DEVERR_PAGE_RANGE);
    }
    const uint32_t n_good = (good & 1) + (good >> 1);
    // a later tile of the run into L2, in whole pages
    const int ahead = lp - base_lp + 2 * kAhead + (lane & 1);
    const int page_cur = __shfl_sync(0xffffffffu, cur, ahead & 31), page_nxt = __shfl_sync(0xffffffffu, nxt, ahead & 31);
    const int page = ahead < 32 ? page_cur : page_nxt;
    if (w.group == 0 && w.t + kAhead < w.to && lane < 2 && page >= 0 && (int64_t)page < p.num_pages)
      ptx::prefetch_l2_bulk(p.kv + (size_t)page * kPageSize * kRecordBytes, kPageSize * kRecordBytes);
    SMLA_WAIT(&bars->scempty[sc.slot], sc.parity ^ 1);
    if (ok && ptx::elect_one()) {
      bars->pages_ok[sc.slot] = good;
      ++bars->armed_sc[sc.slot];
      ptx::mbar_arrive_expect_tx(&bars->scfull[sc.slot], n_good * 1024);
      for (int h = 0; h < 2; ++h)
        if (good >> h & 1)
          ptx::tma_load_3d(base + C::kScale + sc.slot * 2048 + h * 1024, smap, kDLatent, 0, pg[h], &bars->scfull[sc.slot]);
    }
    __syncwarp();
    sc.next();
#pragma unroll 1
    for (int c = 0; c < kChunks; ++c) {
      SMLA_WAIT(&bars->kempty[k.slot], k.parity ^ 1);
      if (ok && ptx::elect_one()) {
        ++bars->armed_k[k.slot];
        ptx::mbar_arrive_expect_tx(&bars->kfull[k.slot], n_good * (kSlot / 2));
        for (int h = 0; h < 2; ++h)
          if (good >> h & 1)
            ptx::tma_load_3d(base + C::kK + k.slot * kSlot + h * (kSlot / 2), map, c < 4 ? 128 * c : kDLatent + 16, 0, pg[h],
                             &bars->kfull[k.slot]);
      }
      __syncwarp();
      k.next();
    }
    w.next(p);
  }
}

template <int NR>
__device__ void mma_role(const WeightsParams& p, uint32_t base, uint32_t tmem, Bars* bars) {
  using C = WC<NR>;
  constexpr uint32_t kIdescCodes = ptx::idesc_e4m3(128, C::kCols), kIdescRope = ptx::idesc_bf16(128, NR);
  Walk w(bars);
  Ring<C::kRing> k;
  Ring<C::kSBufs> s;
  uint32_t qpar = 0, ok = p.wait_ns >= kLeastWaitNs;
  int req = -1, group = -1;
  const uint64_t dq = ptx::sw128_desc(base, 16, 1024), dr = ptx::sw128_desc(base + C::kQr, 16, 1024);
#pragma unroll 1
  while (w.here(p)) {
    if (req != w.req || group != w.group) {
      req = w.req;
      group = w.group;
      SMLA_WAIT(&bars->qfull, qpar);
      qpar ^= 1;
    }
    // (no branch where MMAs are issued: with operands in uniform registers an MMA of N = 64 takes 48 cycles, else 75)
#pragma unroll 1
    for (uint32_t c = 0; c < 4; ++c) {
      SMLA_WAIT(&bars->sempty[s.slot], s.parity ^ 1);
      SMLA_WAIT(&bars->kfull[k.slot], k.parity);
      ptx::tc_fence_after();
      const uint32_t ks = k.slot, ss = s.slot;
      if (ok && ptx::elect_one()) {
        const uint32_t d = tmem + C::kCols * ss;
        const uint64_t dk = ptx::sw128_desc(base + C::kK + ks * kSlot, 16, 1024);
        const uint64_t dqb = dq + (uint64_t)((c * C::kQ8Chunk) >> 4);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
#pragma unroll
          for (int pass = 0; pass < C::kPasses; ++pass)
            ptx::mma_f8_ss(d, dk + 2 * kk, dqb + 2 * kk + (uint64_t)((pass * NR * 128) >> 4), kIdescCodes, kk > 0 || pass > 0);
        ptx::mma_commit(&bars->kempty[ks]);
        ptx::mma_commit(&bars->sfull[ss]);
      }
      __syncwarp();
      k.next();
      s.next();
    }
    SMLA_WAIT(&bars->sempty[s.slot], s.parity ^ 1);
    SMLA_WAIT(&bars->kfull[k.slot], k.parity);
    ptx::tc_fence_after();
    const uint32_t ks = k.slot, ss = s.slot;
    if (ok && ptx::elect_one()) {
      const uint32_t d = tmem + C::kCols * ss;
      const uint64_t dk = ptx::sw128_desc(base + C::kK + ks * kSlot, 16, 1024);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) ptx::mma_f16_ss(d, dk + 2 * kk, dr + 2 * kk, kIdescRope, kk > 0);
      ptx::mma_commit(&bars->kempty[ks]);
      ptx::mma_commit(&bars->sfull[ss]);
    }
    __syncwarp();
    k.next();
    s.next();
    w.next(p);
  }
  if (ptx::elect_one()) ptx::mma_commit(&bars->drain);
  __syncwarp();
}

// Rows of one group into the Q operands; factors, -lse log2 e and lengths to buffer `buf`.  A warp takes rows warp,
// warp + 8, ..., two at a time.
template <int NR>
__device__ __forceinline__ void load_q(const WeightsParams& p, int req, int group, unsigned char* sm, uint32_t base, int buf,
                                       int warp, int lane) {
  using C = WC<NR>;
  const int row0 = group * NR, nrows = min(NR, p.q_per_req * p.H - row0);
  const size_t first = (size_t)req * p.q_per_req * p.H + row0;         // of all (query, head) rows
  float* f = reinterpret_cast<float*>(sm + C::kRows) + buf * 3 * NR;
  const int b = lane >> 3, u = lane & 7;
#pragma unroll 2
  for (int i = 0; i < NR / kSoftWarps; ++i) {
    const int r = warp + kSoftWarps * i;
    const uint4* src = reinterpret_cast<const uint4*>(p.q + (first + r) * kDQK);
    uint4 a = make_uint4(0u, 0u, 0u, 0u), c = a, rope = a;
    float lse = 0.f;
    int len = 0;
    if (r < nrows) {
      a = __ldg(src + 2 * lane);
      c = __ldg(src + 2 * lane + 1);
      if (lane < 8) rope = __ldg(src + 64 + lane);
      lse = __ldg(p.lse + first + r);
      len = clamped_len(p, req * p.q_per_req + (row0 + r) / p.H);
    }
    const uint32_t wds[8] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
    uint32_t hi[4], lo[4];
    const int x = split_q(wds, hi, lo);
    const uint32_t q8 = base + b * C::kQ8Chunk;
    ptx::sts128(q8 + swz128(r, u), make_uint4(hi[0], hi[1], hi[2], hi[3]));
    ptx::sts128(q8 + swz128(NR + r, u), make_uint4(lo[0], lo[1], lo[2], lo[3]));
    if (lane < 8) ptx::sts128(base + C::kQr + swz128(r, lane), rope);
    if (lane == 0) {
      f[r] = exp2_int(x) * (p.sm_scale * kLog2e);
      f[NR + r] = lse == -CUDART_INF_F ? lse : -lse * kLog2e;      // a row that saw nothing adds nothing
      reinterpret_cast<int*>(f)[2 * NR + r] = len;
    }
  }
}

template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t a, uint32_t (&r)[N]) {
  if constexpr (N == 32) ptx::tmem_ld32(a, r);
  else if constexpr (N == 16) ptx::tmem_ld16(a, r);
  else ptx::tmem_ld8(a, r);
}

template <int NR>
__device__ void softmax_role(const WeightsParams& p, unsigned char* sm, uint32_t base, uint32_t tmem, Bars* bars, int warp,
                             int lane) {
  using C = WC<NR>;
  constexpr int HC = C::HC, kStep = HC < 32 ? HC : 32;      // rows read at once
  const int part = warp >> 2, quad = warp & 3, col0 = part * HC, tok = 32 * quad + lane;
  const uint32_t lane_base = tmem + ((uint32_t)(32 * quad) << 16);
  const float kf = p.sm_scale * kLog2e;
  Walk w(bars);
  Ring<C::kSBufs> s;
  Ring<C::kScaleSlots> sc;
  uint32_t ok = p.wait_ns >= kLeastWaitNs;
  int req = -1, group = -1, buf = 0, flip = 0, shortest = 0;
#pragma unroll 1
  while (w.here(p)) {
    if (req != w.req || group != w.group) {
      // every score of the tiles before has been computed (this warp waited for the last), so no MMA reads the old rows
      req = w.req;
      group = w.group;
      buf ^= 1;
      load_q<NR>(p, req, group, sm, base, buf, warp, lane);
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (ok && lane == 0) ptx::mbar_arrive(&bars->qfull);
      shortest = 0x7fffffff;
      const int b0 = req * p.q_per_req;
      const int last = min((group + 1) * NR, p.q_per_req * p.H) - 1;
#pragma unroll 1
      for (int b = b0 + group * NR / p.H; b <= b0 + last / p.H; ++b) shortest = min(shortest, clamped_len(p, b));
      ptx::named_bar_sync(1, kSoftWarps * 32);              // the rows' factors are written
    }
    const int t = w.t * kDenseTile + tok;                   // (tiles begin below cols, which is below 2^30)
    const bool mine = part == 0 && t < w.len;
    float* at = p.weights + (size_t)w.req * p.weights_stride + t;
    float old = 0.f;
    if (mine && (w.group > 0 || p.decay != 0.f)) old = *at;
    SMLA_WAIT(&bars->scfull[sc.slot], sc.parity);
    const float4 s4 = ptx::lds128f(base + C::kScale + sc.slot * 2048 + tok * 16);
    const int pages = bars->pages_ok[sc.slot];
    __syncwarp();
    if (ok && lane == 0) ptx::mbar_arrive(&bars->scempty[sc.slot]);
    sc.next();
    uint64_t acc[HC / 2];                                   // pairs of rows
#pragma unroll
    for (int i = 0; i < HC / 2; ++i) acc[i] = 0;
    {
      float4 rot = s4;
#pragma unroll 1
      for (int b = 0; b < 4; ++b) {
        SMLA_WAIT(&bars->sfull[s.slot], s.parity);
        ptx::tc_fence_after();
        const uint32_t a = lane_base + C::kCols * s.slot + col0;
        const uint64_t scale = ptx::pack2(rot.x, rot.x);
        rot = make_float4(rot.y, rot.z, rot.w, rot.x);
#pragma unroll
        for (int i0 = 0; i0 < HC; i0 += kStep) {
          uint32_t x[kStep], y[kStep];
          tmem_ld<kStep>(a + i0, x);
          if constexpr (C::kPasses == 1) tmem_ld<kStep>(a + NR + i0, y);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < kStep; i += 2) {
            uint64_t v = ptx::pack2(x[i], x[i + 1]);
            if constexpr (C::kPasses == 1) v = ptx::add2(v, ptx::pack2(y[i], y[i + 1]));
            acc[(i0 + i) / 2] = ptx::fma2(v, scale, acc[(i0 + i) / 2]);
          }
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (ok && lane == 0) ptx::mbar_arrive(&bars->sempty[s.slot]);
        s.next();
      }
    }
    // exponents: 2^x sm_scale log2 e (latent part) + (sm_scale log2 e (rope part) - lse log2 e)
    SMLA_WAIT(&bars->sfull[s.slot], s.parity);
    ptx::tc_fence_after();
    const uint32_t rows = base + C::kRows + (buf * 3 * NR + col0) * 4;
    uint64_t sum2[2] = {0, 0};
    const bool all = (long long)(w.t + 1) * kDenseTile <= shortest && (group + 1) * NR <= p.q_per_req * p.H;
#pragma unroll
    for (int i0 = 0; i0 < HC; i0 += kStep) {
      uint32_t x[kStep];
      tmem_ld<kStep>(lane_base + C::kCols * s.slot + col0 + i0, x);
      ptx::tmem_wait_ld();
      const uint64_t kf2 = ptx::pack2(kf, kf);
#pragma unroll
      for (int i = 0; i < kStep; i += 4) {
        const ulonglong2 f = ptx::lds128_pairs(rows + (i0 + i) * 4), l = ptx::lds128_pairs(rows + (NR + i0 + i) * 4);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 d = ptx::unpack2(ptx::fma2(acc[(i0 + i) / 2 + j], j ? f.y : f.x,
                                                  ptx::fma2(ptx::pack2(x[i + 2 * j], x[i + 2 * j + 1]), kf2, j ? l.y : l.x)));
          float a = ptx::ex2_approx(d.x), b = ptx::ex2_approx(d.y);
          if (!all) {                                       // rows that do not see the position, and rows that are none
            const int* lens = reinterpret_cast<const int*>(sm + C::kRows) + (buf * 3 + 2) * NR + col0 + i0 + i + 2 * j;
            if (t >= lens[0]) a = 0.f;
            if (t >= lens[1]) b = 0.f;
          }
          sum2[j] = ptx::add2(sum2[j], ptx::pack2(a, b));
        }
      }
    }
    ptx::tc_fence_before();
    __syncwarp();
    if (ok && lane == 0) ptx::mbar_arrive(&bars->sempty[s.slot]);
    s.next();
    const float2 e = ptx::unpack2(ptx::add2(sum2[0], sum2[1]));
    float sum = e.x + e.y;
    const uint32_t meet = base + C::kSum + (flip * 128 + tok) * 4;
    if (part == 1) ptx::sts32f(meet, sum);
    ptx::named_bar_sync(1, kSoftWarps * 32);
    flip ^= 1;
    if (mine && ok) {
      sum += ptx::lds32f(meet);
      if (!(pages >> (tok >> 6) & 1)) sum = 0.f;            // a position whose record is not in the cache
      *at = w.group > 0 ? old + sum : p.decay != 0.f ? fmaf(p.decay, old, sum) : sum;
    }
    w.next(p);
  }
}

// This CTA's run of tiles [T c / n, T (c + 1) / n) of all requests' tiles laid end to end.
__device__ __forceinline__ void find_run(const WeightsParams& p, Bars* bars) {
  const int n = p.requests, per = (n + kThreads - 1) / kThreads, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i0 = min(n, (int)threadIdx.x * per), i1 = min(n, i0 + per);
  long long mine = 0;
#pragma unroll 1
  for (int i = i0; i < i1; ++i) mine += tiles_of(longest(p, i));
  long long upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += up;
  }
  if (lane == 31) bars->sums[warp] = upto;
  if (threadIdx.x == 0) bars->run = bars->first_req = bars->first_tile = 0;
  __syncthreads();
  long long total = 0, before = upto - mine;
#pragma unroll 1
  for (int x = 0; x < kThreads / 32; ++x) {
    total += bars->sums[x];
    if (x < warp) before += bars->sums[x];
  }
  const long long a = total * blockIdx.x / gridDim.x, e = total * (blockIdx.x + 1) / gridDim.x;
  if (a < e && before <= a && a < before + mine) {           // the run begins in one of this thread's requests
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
      const int tiles = tiles_of(longest(p, i));
      if (a < before + tiles) {
        bars->first_req = i;
        bars->first_tile = (int)(a - before);
        bars->run = (int)(e - a);
        break;
      }
      before += tiles;
    }
  }
  __syncthreads();
}

template <int NR>
__global__ void __launch_bounds__(kThreads, 1)
    weights_kernel(const WeightsParams p, const __grid_constant__ CUtensorMap map, const __grid_constant__ CUtensorMap smap) {
  using C = WC<NR>;
  extern __shared__ __align__(1024) unsigned char sm[];
  const uint32_t base = ptx::smem_u32(sm);
  Bars* bars = reinterpret_cast<Bars*>(sm + C::kBar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == kCopyWarp) {
    constexpr int kBars = offsetof(Bars, tmem) / 8;
    constexpr uint64_t kBySoftmax = (31ull << offsetof(Bars, sempty) / 8) | (7ull << offsetof(Bars, scempty) / 8) |
                                    (1ull << offsetof(Bars, qfull) / 8);
    static_assert(kBars <= 64, "one bit per barrier");
    for (int i = lane; i < kBars; i += 32)
      ptx::mbar_init(reinterpret_cast<uint64_t*>(bars) + i, kBySoftmax >> i & 1 ? kSoftWarps : 1);
    if (lane < 10) bars->armed_k[lane] = 0;
    if (lane < 3) bars->armed_sc[lane] = 0;
    if (lane == 0) {
      bars->abort = p.wait_ns < kLeastWaitNs;
      ptx::prefetch_tensormap(&map);
      ptx::prefetch_tensormap(&smap);
    }
    ptx::fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(&bars->tmem, C::kTmemCols);
    ptx::tmem_relinquish();
  }
  find_run(p, bars);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = bars->tmem;

  if (warp < kSoftWarps) softmax_role<NR>(p, sm, base, tmem, bars, warp, lane);
  else if (warp == kCopyWarp) copy_role<NR>(p, &map, &smap, base, bars, lane);
  else mma_role<NR>(p, base, tmem, bars);

  // nothing of this CTA's may be in flight when it leaves
  ptx::tc_fence_before();
  __syncthreads();
  int never = 0;
  if (warp == kCopyWarp && bars->abort) {
    drain_copies(bars->kfull, bars->armed_k, C::kRing, lane);
    drain_copies(bars->scfull, bars->armed_sc, C::kScaleSlots, lane);
  }
  if (warp == kMmaWarp) {
    ptx::mbar_wait_warp(&bars->drain, 0, &never, lane, 100000000ull);
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::kTmemCols);
  }
  if (threadIdx.x == 0 && bars->abort && p.err) atomicOr(p.err, SMLA_DEVERR_TIMEOUT);
}

// Without columns there are no tiles: the lengths alone are looked at.
__global__ void __launch_bounds__(kThreads) lengths_kernel(const WeightsParams p) {
  bool over = false;
  for (int b = threadIdx.x; b < p.requests * p.q_per_req; b += kThreads) over |= __ldg(p.seq_lens + b) > clamped_len(p, b);
  if (over) atomicOr(p.err, SMLA_DEVERR_LEN_RANGE);
}

template <int NR>
cudaError_t launch_nr(const WeightsParams& p, int ctas, cudaStream_t stream) {
  CUtensorMap map, smap;
  if (!encoder() || !encode_map(&map, p.kv, p.num_pages, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_map(&smap, p.kv, p.num_pages, 16, CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorNotSupported;
  static std::atomic<bool> set[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !set[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(weights_kernel<NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, WC<NR>::kBytes);
    if (e != cudaSuccess) return e;
    if (dev < 64) set[dev].store(true, std::memory_order_relaxed);
  }
  weights_kernel<NR><<<ctas, kThreads, WC<NR>::kBytes, stream>>>(p, map, smap);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_weights(const WeightsParams& q, int sms, cudaStream_t stream) {
  if (q.requests == 0) return cudaSuccess;
  if (q.cols == 0) {
    if (q.err && q.seq_lens) lengths_kernel<<<1, kThreads, 0, stream>>>(q);
    return cudaGetLastError();
  }
  WeightsParams p = q;
  const long long rows = (long long)p.q_per_req * p.H;
  const int nr = rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
  p.groups = (int)((rows + nr - 1) / nr);
  const long long slots = (long long)p.max_pages * kPageSize < p.cols ? (long long)p.max_pages * kPageSize : p.cols;
  const long long most = p.requests * ((slots + kDenseTile - 1) / kDenseTile);
  const int ctas = (int)(most < sms ? most : sms);
  if (nr == 16) return launch_nr<16>(p, ctas, stream);
  if (nr == 32) return launch_nr<32>(p, ctas, stream);
  if (nr == 64) return launch_nr<64>(p, ctas, stream);
  return launch_nr<128>(p, ctas, stream);
}

}  // namespace smla
