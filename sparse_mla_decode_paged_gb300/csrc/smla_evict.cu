// Eviction from the paged cache by accumulated attention weight, in place.
//
// Of a request's n = seq_lens[r] records the k = min(n, max(keep, held)) first in this order stay: the held ones (position
// below `sinks`, or among the `recent` positions before next_positions[r]), then by weight (IEEE totalOrder), then the lower
// slot.  The survivors at slots >= k move, in slot order, to the free slots below k: every source is at or past k and
// every destination below, so all records move at once, and no others are read or written.  (Keeping the order of the
// slots would move nearly every record behind the first free slot; scores do not depend on it, the rotation being in
// the records.)  Weights and positions move along; the weights of slots k .. n - 1 become 0.
//
// Select: a cluster of 1 .. 8 CTAs per request, each warp with a contiguous part of the slots.  The k-th largest key by
// histograms of 11, 11 and 10 bits, summed over the cluster through distributed shared memory; then every warp counts
// its ties, free slots and survivors, and writes its part of the two lists behind those of the warps before it.  Keys
// stay in shared memory.  Move: one warp per record, two in flight.
// What bounds it: the selection is a chain of cluster barriers and passes over shared memory, the moves HBM bytes.
#include <cuda_runtime.h>

#include <atomic>

#include "smla_device.cuh"
#include "smla_internal.h"
#include "smla_ptx.cuh"

namespace smla {
namespace {

constexpr int kWarps = 32;
constexpr int kThreads = 32 * kWarps;
constexpr int kMostCluster = 8;
constexpr int kBins = 2048;
constexpr int kKeySlots = 40960;          // slots of a CTA whose keys fit into shared memory
constexpr int kSlotsPerCta = 4096;        // a request takes another CTA per so many slots
constexpr uint32_t kDynBytes = kKeySlots * 4 + kKeySlots / 8;

struct Shared {
  uint32_t hist[3][kBins];
  uint32_t scan[kWarps];
  uint32_t held;                          // of this CTA
  uint32_t ties[kWarps];                  // of each warp
  uint2 moves[kWarps];                    // free slots and survivors of each warp
  uint32_t digit, above;
};

__device__ __forceinline__ uint32_t ld_cluster(const void* local, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(ptx::mapa(ptx::smem_u32(local), rank)) : "memory");
  return v;
}

// The order of the values as unsigned numbers.
__device__ __forceinline__ uint32_t order_key(float w) {
  const uint32_t b = __float_as_uint(w);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ uint32_t warp_sum(uint32_t v) { return __reduce_add_sync(0xffffffffu, v); }

// Slots of a request.
__device__ __forceinline__ int length_of(const EvictParams& p, int r) {
  const long long most = min((long long)p.cols, (long long)p.max_pages * kPageSize);
  return (int)min((long long)max(__ldcg(p.seq_lens + r), 0), most);
}

__global__ void __launch_bounds__(kThreads, 1) evict_select_kernel(const EvictParams p, int csize) {
  extern __shared__ __align__(16) uint32_t dyn[];
  __shared__ Shared s;
  uint32_t* keys = dyn;
  uint32_t* heldbits = dyn + kKeySlots;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = blockIdx.x / csize;
  const uint32_t rank = csize > 1 ? ptx::cluster_ctarank() : 0;
  if (threadIdx.x == 0) ptx::griddep_launch_dependents();
  const int n = length_of(p, r);
  const int keep = max(p.keep ? __ldg(p.keep + r) : p.keep_all, 0);
  // in 64 bits: positions and `recent` may be anywhere in their type
  const long long recent_from = (long long)__ldg(p.next_positions + r) - p.recent;
  const int per = (int)(((long long)n + (long long)csize * kThreads - 1) / ((long long)csize * kThreads)) * 32;   // per warp
  const int t0 = (int)min((long long)n, (long long)((int)rank * kWarps + warp) * per), t1 = min(n, t0 + per);
  const int first = (int)min((long long)n, (long long)rank * kWarps * per);          // of the CTA
  const bool cached = per * kWarps <= kKeySlots;
  float* w = p.weights + (size_t)r * p.weights_stride;
  const int32_t* pos = p.positions + (size_t)r * p.positions_stride;
  if (threadIdx.x == 0 && rank == 0 && p.err && __ldcg(p.seq_lens + r) > n) atomicOr(p.err, SMLA_DEVERR_LEN_RANGE);

  auto sync = [&]() {
    if (csize > 1) ptx::cluster_sync_all();
    else __syncthreads();
  };
  // key of slot t, and whether it is held
  auto load = [&](int t, bool& held) -> uint32_t {
    if (cached) {
      held = heldbits[(t - first) >> 5] >> (t - first & 31) & 1;
      return keys[t - first];
    }
    const int at = __ldg(pos + t);
    held = at < p.sinks || at >= recent_from;
    return order_key(w[t]);
  };

  for (int i = threadIdx.x; i < 3 * kBins; i += kThreads) (&s.hist[0][0])[i] = 0;
  if (threadIdx.x == 0) s.held = 0;
  __syncthreads();
  uint32_t mine = 0;
#pragma unroll 4
  for (int b = t0; b < t1; b += 32) {
    const int t = b + lane;
    const bool in = t < t1;
    uint32_t key = 0;
    bool held = false;
    if (in) {
      const int at = __ldg(pos + t);
      key = order_key(w[t]);
      held = at < p.sinks || at >= recent_from;
      if (!held) atomicAdd(&s.hist[0][key >> 21], 1u);
    }
    const uint32_t bits = __ballot_sync(0xffffffffu, held);
    mine += __popc(bits);
    if (cached) {
      if (in) keys[t - first] = key;
      if (lane == 0) heldbits[(b - first) >> 5] = bits;
    }
  }
  if (lane == 0 && mine) atomicAdd(&s.held, mine);
  sync();
  uint32_t held_all = 0;
  for (int c = 0; c < csize; ++c) held_all += ld_cluster(&s.held, c);
  const int k = min(n, max(keep, (int)held_all));
  int32_t* lists = p.lists + (size_t)r * 2 * p.list_len;               // free slots, then survivors
  if (k == n) {                                                       // (the same in every CTA of the cluster)
    sync();                                                           // the other CTAs have read this one's count
    if (threadIdx.x == 0 && rank == 0) {
      p.moved[r] = 0;
      p.new_lens[r] = n;
    }
    return;
  }
  // the key from which on records stay: `need` of those that are not held
  uint32_t need = (uint32_t)k - held_all, limit = 0, ties = 0;
  const bool some = need > 0;
  if (some) {
#pragma unroll 1
    for (int d = 0; d < 3; ++d) {
      const int shift = d == 0 ? 21 : d == 1 ? 10 : 0, bins = d == 2 ? 1024 : kBins;
      if (d > 0) {
#pragma unroll 4
        for (int b = t0; b < t1; b += 32) {
          const int t = b + lane;
          if (t >= t1) continue;
          bool held;
          const uint32_t key = load(t, held);
          if (!held && key >> (shift + (d == 2 ? 10 : 11)) == limit) atomicAdd(&s.hist[d][key >> shift & (bins - 1)], 1u);
        }
        sync();
      }
      // bins from the top: thread i has 2 i and 2 i + 1 of them
      uint32_t c[2] = {0, 0};
      const int top = bins - 1 - 2 * (int)threadIdx.x;
      if (top >= 0)
        for (int x = 0; x < csize; ++x) {
          c[0] += ld_cluster(&s.hist[d][top], x);
          c[1] += ld_cluster(&s.hist[d][top - 1], x);
        }
      uint32_t upto = c[0] + c[1];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t up = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += up;
      }
      if (lane == 31) s.scan[warp] = upto;
      __syncthreads();
      uint32_t before = lane < warp ? s.scan[lane] : 0;
      before = warp_sum(before) + upto - c[0] - c[1];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (before < need && need <= before + c[j]) {
          s.digit = (uint32_t)(top - j);
          s.above = before;
          s.ties[0] = c[j];
        }
        before += c[j];
      }
      __syncthreads();
      limit = limit << (d == 2 ? 10 : 11) | s.digit;
      need -= s.above;
      ties = s.ties[0];
      __syncthreads();
    }
  }
  // the first `need` slots whose key is the limit stay: ties of the warps before this one
  uint32_t tie = 0;
  if (some && need < ties) {
    uint32_t m = 0;
    for (int b = t0; b < t1; b += 32) {
      bool held = true;
      const uint32_t key = b + lane < t1 ? load(b + lane, held) : 0u;
      m += __popc(__ballot_sync(0xffffffffu, !held && key == limit));
    }
    if (lane == 0) s.ties[warp] = m;
    sync();
    uint32_t x = 0;
    for (int c = 0; c <= (int)rank; ++c)
      if (c < (int)rank || lane < warp) x += ld_cluster(&s.ties[lane], c);
    tie = warp_sum(x);
  }
  // which of a step's 32 slots stay
  uint32_t seen = tie;
  auto stays = [&](int b) -> uint32_t {
    bool held = true;
    const bool in = b + lane < t1;
    const uint32_t key = in ? load(b + lane, held) : 0u;
    const uint32_t same = __ballot_sync(0xffffffffu, some && !held && key == limit);
    const bool first_ones = seen + __popc(same & ((1u << lane) - 1u)) < need;
    seen += __popc(same);
    return __ballot_sync(0xffffffffu, in && (held || (some && (key > limit || (key == limit && first_ones)))));
  };
  // slots of a step that are free below k, and that survive at or past it
  auto below_k = [&](int b) -> uint32_t { return b + 32 <= k ? ~0u : b >= k ? 0u : (1u << (k - b)) - 1u; };
  auto inside = [&](int b) -> uint32_t { return b + 32 <= t1 ? ~0u : (1u << (t1 - b)) - 1u; };
  uint2 m = make_uint2(0u, 0u);
  for (int b = t0; b < t1; b += 32) {
    const uint32_t kept = stays(b);
    m.x += __popc(~kept & below_k(b) & inside(b));
    m.y += __popc(kept & ~below_k(b));
  }
  if (lane == 0) s.moves[warp] = m;
  sync();
  uint32_t x = 0, y = 0, all = 0;
  for (int c = 0; c < csize; ++c) {
    const uint32_t f = ld_cluster(&s.moves[lane].x, c), g = ld_cluster(&s.moves[lane].y, c);
    if (c < (int)rank || (c == (int)rank && lane < warp)) x += f, y += g;
    all += g;
  }
  x = warp_sum(x);
  y = warp_sum(y);
  all = warp_sum(all);
  seen = tie;
  const uint32_t lower = (1u << lane) - 1u;
  for (int b = t0; b < t1; b += 32) {
    const uint32_t kept = stays(b), low = below_k(b), free = ~kept & low & inside(b), moves = kept & ~low;
    const int t = b + lane;
    if (free >> lane & 1) lists[x + __popc(free & lower)] = t;
    if (moves >> lane & 1) lists[p.list_len + y + __popc(moves & lower)] = t;
    if (t < t1 && !(low >> lane & 1) && !(kept >> lane & 1)) w[t] = 0.f;
    x += __popc(free);
    y += __popc(moves);
  }
  if (threadIdx.x == 0 && rank == 0) {
    p.moved[r] = (int32_t)all;
    p.new_lens[r] = k;
  }
  sync();                                               // nobody leaves while its shared memory is read
}

// ----------------------------------------------------------------------------- move

constexpr int kMoveThreads = 256;
constexpr int kUnits = kRecordBytes / 16;               // 41
constexpr int kPairs = 2;                               // records in flight per warp

__device__ __forceinline__ unsigned char* record(const EvictParams& p, int r, int t) {
  const int page = __ldg(p.block_table + (size_t)r * p.max_pages + (t >> 6));
  return page >= 0 && (int64_t)page < p.num_pages
             ? p.kv + ((int64_t)page * kPageSize + (t & (kPageSize - 1))) * kRecordBytes
             : nullptr;
}

// (This grid is resident while the selection still writes, so the lists are read from L2.)
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams p) {
  const int lane = threadIdx.x & 31, r = blockIdx.y;
  ptx::griddep_wait();
  const int moved = __ldcg(p.moved + r), step = gridDim.x * (kMoveThreads / 32) * kPairs;
  const int32_t* lists = p.lists + (size_t)r * 2 * p.list_len;
  float* w = p.weights + (size_t)r * p.weights_stride;
  int32_t* pos = p.positions + (size_t)r * p.positions_stride;
  for (int i = (blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5)) * kPairs; i < moved; i += step) {
    unsigned char *from[kPairs], *to[kPairs];
    int src[kPairs], dst[kPairs];
    uint4 a[kPairs], b[kPairs];
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      from[j] = to[j] = nullptr;
      src[j] = dst[j] = 0;
      if (i + j >= moved) continue;
      dst[j] = __ldcg(lists + i + j);
      src[j] = __ldcg(lists + p.list_len + i + j);
      from[j] = record(p, r, src[j]);
      to[j] = record(p, r, dst[j]);
    }
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      if (!from[j] || !to[j]) continue;
      a[j] = __ldcg(reinterpret_cast<const uint4*>(from[j]) + lane);
      if (lane < kUnits - 32) b[j] = __ldcg(reinterpret_cast<const uint4*>(from[j]) + 32 + lane);
    }
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      if (i + j >= moved) continue;
      if (lane == 0) {
        w[dst[j]] = __ldcg(w + src[j]);
        w[src[j]] = 0.f;
        pos[dst[j]] = __ldcg(pos + src[j]);
      }
      if (!from[j] || !to[j]) {
        if (lane == 0 && p.err) atomicOr(p.err, SMLA_DEVERR_PAGE_RANGE);
        continue;
      }
      reinterpret_cast<uint4*>(to[j])[lane] = a[j];
      if (lane < kUnits - 32) reinterpret_cast<uint4*>(to[j])[32 + lane] = b[j];
    }
  }
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, int sms, cudaStream_t stream) {
  if (p.requests == 0) return cudaSuccess;
  static std::atomic<bool> set[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !set[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kDynBytes);
    if (e != cudaSuccess) return e;
    if (dev < 64) set[dev].store(true, std::memory_order_relaxed);
  }
  // one CTA per kSlotsPerCta slots, while the requests leave SMs for them
  int csize = 1;
  while (csize < kMostCluster && (long long)p.requests * csize * 2 <= sms && p.cols > (long long)csize * kSlotsPerCta)
    csize *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.requests * csize);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kDynBytes;
  cfg.stream = stream;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeClusterDimension;
  a[0].val.clusterDim.x = csize;
  a[0].val.clusterDim.y = a[0].val.clusterDim.z = 1;
  cfg.attrs = a;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, evict_select_kernel, p, csize);
  if (e != cudaSuccess) return e;
  const int warps = kMoveThreads / 32;
  long long blocks = ((long long)p.list_len + warps * kPairs - 1) / (warps * kPairs);
  const long long fill = ((long long)sms * 8 + p.requests - 1) / p.requests;
  if (blocks > fill) blocks = fill;
  cudaLaunchConfig_t mv = {};
  mv.gridDim = dim3((unsigned)(blocks < 1 ? 1 : blocks), (unsigned)p.requests);
  mv.blockDim = dim3(kMoveThreads);
  mv.stream = stream;
  cudaLaunchAttribute b[1];
  b[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  b[0].val.programmaticStreamSerializationAllowed = 1;
  mv.attrs = b;
  mv.numAttrs = 1;
  return cudaLaunchKernelEx(&mv, evict_move_kernel, p);
}

}  // namespace smla
