// Eviction from the paged cache by accumulated attention weight, in place.
//
// Of a request's n = seq_lens[r] records the k = min(n, max(keep, held)) first in this order stay: the held ones (position
// below `sinks`, or among the `recent` positions before next_positions[r]), then by weight (IEEE totalOrder), then the lower
// slot.  The survivors at slots >= k move, in slot order, to the free slots below k: every source is at or past k and
// every destination below, so all records move at once, and no others are read or written.  (Keeping the order of the
// slots would move nearly every record behind the first free slot; scores do not depend on it, the rotation being in
// the records.)  Weights and positions move along; the weights of slots k .. n - 1 become 0.
//
// Select: a cluster of 1 .. 16 CTAs per request, each warp with a contiguous part of the slots.  The k-th largest key by
// histograms of 11, 11 and 10 bits, summed over the cluster through distributed shared memory; then every warp counts
// its ties, free slots and survivors, and writes its part of the two lists behind those of the warps before it.  Keys
// stay in shared memory.  Move: a warp has four records in flight.
// What bounds it: the selection is a chain of cluster barriers and passes over shared memory, the moves HBM bytes.
#include <cuda_runtime.h>

#include <atomic>

#include "smla_device.cuh"
#include "smla_evict_plan.h"
#include "smla_internal.h"
#include "smla_ptx.cuh"

namespace smla {
namespace {

constexpr int kWarps = 32;
constexpr int kThreads = 32 * kWarps;
constexpr int kBins = 2048;
constexpr int kBatch = 4;                 // steps of 32 slots that a warp loads at once
constexpr int kKeySlots = kEvictKeySlots;
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
  // keys of kBatch steps of 32 slots from b on, one per lane, and their held slots (a bit each): all loads first
  struct Keys {
    uint32_t key[kBatch], held[kBatch];
  };
  auto load = [&](int b) {
    Keys k;
    if (cached) {
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int at = b + 32 * j - first;
        k.key[j] = b + 32 * j + lane < t1 ? keys[at + lane] : 0u;
        k.held[j] = b + 32 * j < t1 ? heldbits[at >> 5] : 0u;
      }
    } else {
      float v[kBatch];
      int at[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int t = b + 32 * j + lane;
        v[j] = t < t1 ? __ldcg(w + t) : 0.f;
        at[j] = t < t1 ? __ldg(pos + t) : 0;
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const bool in = b + 32 * j + lane < t1;
        k.key[j] = order_key(v[j]);
        k.held[j] = __ballot_sync(0xffffffffu, in && (at[j] < p.sinks || at[j] >= recent_from));
      }
    }
    return k;
  };

  for (int i = threadIdx.x; i < 3 * kBins; i += kThreads) (&s.hist[0][0])[i] = 0;
  if (threadIdx.x == 0) s.held = 0;
  __syncthreads();
  uint32_t mine = 0;
#pragma unroll 1
  for (int b0 = t0; b0 < t1; b0 += 32 * kBatch) {
    float v[kBatch];
    int at[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int t = b0 + 32 * j + lane;
      v[j] = t < t1 ? __ldcg(w + t) : 0.f;
      at[j] = t < t1 ? __ldg(pos + t) : 0;
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int b = b0 + 32 * j, t = b + lane;
      if (b >= t1) break;
      const bool in = t < t1, held = in && (at[j] < p.sinks || at[j] >= recent_from);
      const uint32_t key = order_key(v[j]), bits = __ballot_sync(0xffffffffu, held);
      if (in && !held) atomicAdd(&s.hist[0][key >> 21], 1u);
      mine += __popc(bits);
      if (cached) {
        if (in) keys[t - first] = key;
        if (lane == 0) heldbits[(b - first) >> 5] = bits;
      }
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
#pragma unroll 1
        for (int b = t0; b < t1; b += 32 * kBatch) {
          const Keys k = load(b);
#pragma unroll
          for (int j = 0; j < kBatch; ++j)
            if (b + 32 * j + lane < t1 && !(k.held[j] >> lane & 1) && k.key[j] >> (shift + (d == 2 ? 10 : 11)) == limit)
              atomicAdd(&s.hist[d][k.key[j] >> shift & (bins - 1)], 1u);
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
      if (need == ties) {                                  // all keys from here on stay, whatever their lower bits
        limit <<= shift;
        break;
      }
    }
  }
  // the first `need` slots whose key is the limit stay: ties of the warps before this one
  uint32_t tie = 0;
  if (some && need < ties) {
    uint32_t m = 0;
#pragma unroll 1
    for (int b = t0; b < t1; b += 32 * kBatch) {
      const Keys k = load(b);
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        m += __popc(__ballot_sync(0xffffffffu, b + 32 * j + lane < t1 && k.key[j] == limit) & ~k.held[j]);
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
  auto stays = [&](int b, uint32_t key, uint32_t held) -> uint32_t {
    const bool in = b + lane < t1;
    const uint32_t same = some ? __ballot_sync(0xffffffffu, in && key == limit) & ~held : 0u;
    const bool first_ones = seen + __popc(same & ((1u << lane) - 1u)) < need;
    seen += __popc(same);
    return held | __ballot_sync(0xffffffffu, in && some && (key > limit || (key == limit && first_ones)));
  };
  // slots of a step that are free below k, and that survive at or past it
  auto below_k = [&](int b) -> uint32_t { return b + 32 <= k ? ~0u : b >= k ? 0u : (1u << (k - b)) - 1u; };
  auto inside = [&](int b) -> uint32_t { return b + 32 <= t1 ? ~0u : (1u << (t1 - b)) - 1u; };
  uint2 m = make_uint2(0u, 0u);
#pragma unroll 1
  for (int b0 = t0; b0 < t1; b0 += 32 * kBatch) {
    const Keys ks = load(b0);
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int b = b0 + 32 * j;
      if (b >= t1) break;
      const uint32_t kept = stays(b, ks.key[j], ks.held[j]);
      m.x += __popc(~kept & below_k(b) & inside(b));
      m.y += __popc(kept & ~below_k(b));
    }
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
#pragma unroll 1
  for (int b0 = t0; b0 < t1; b0 += 32 * kBatch) {
    const Keys ks = load(b0);
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int b = b0 + 32 * j, t = b + lane;
      if (b >= t1) break;
      const uint32_t kept = stays(b, ks.key[j], ks.held[j]), low = below_k(b), free = ~kept & low & inside(b),
                     moves = kept & ~low;
      if (free >> lane & 1) lists[x + __popc(free & lower)] = t;
      if (moves >> lane & 1) lists[p.list_len + y + __popc(moves & lower)] = t;
      if (t < t1 && !(low >> lane & 1) && !(kept >> lane & 1)) w[t] = 0.f;
      x += __popc(free);
      y += __popc(moves);
    }
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
constexpr int kPairs = 4;                               // records in flight per warp

// Slot of a list's entry `lane` (lanes 0 .. 3: free slots, 4 .. 7: survivors) and its record's row in the cache: -1 where its
// page is not in it.
struct Place {
  int slot;
  int64_t row;
};

__device__ __forceinline__ Place place_of(const EvictParams& p, const int32_t* lists, int r, int i, int moved, int lane) {
  Place x{0, -1};
  const int at = i + (lane & (kPairs - 1));
  if (lane >= 2 * kPairs || at >= moved) return x;
  x.slot = __ldcg(lists + (lane < kPairs ? at : p.list_len + at));
  const int page = __ldg(p.block_table + (size_t)r * p.max_pages + (x.slot >> 6));
  if (page >= 0 && (int64_t)page < p.num_pages) x.row = (int64_t)page * kPageSize + (x.slot & (kPageSize - 1));
  return x;
}

// A warp moves kPairs records at a time, their places looked up while the ones before are under way.  (This grid is resident
// while the selection still writes, so the lists are read from L2.)
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams p) {
  const int lane = threadIdx.x & 31, r = blockIdx.y;
  ptx::griddep_wait();
  const int moved = __ldcg(p.moved + r), step = gridDim.x * (kMoveThreads / 32) * kPairs;
  const int32_t* lists = p.lists + (size_t)r * 2 * p.list_len;
  float* w = p.weights + (size_t)r * p.weights_stride;
  int32_t* pos = p.positions + (size_t)r * p.positions_stride;
  int i = (blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5)) * kPairs;
  Place next = place_of(p, lists, r, i, moved, lane);
#pragma unroll 1
  for (; i < moved; i += step) {
    const Place here = next;
    uint4 a[kPairs], b[kPairs];
    const unsigned char* from[kPairs];
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      const int64_t dst = __shfl_sync(0xffffffffu, here.row, j), src = __shfl_sync(0xffffffffu, here.row, kPairs + j);
      from[j] = dst >= 0 && src >= 0 ? p.kv + src * kRecordBytes : nullptr;
      if (!from[j]) continue;
      a[j] = __ldcg(reinterpret_cast<const uint4*>(from[j]) + lane);
      if (lane < kUnits - 32) b[j] = __ldcg(reinterpret_cast<const uint4*>(from[j]) + 32 + lane);
    }
    // weights and positions: lane j for pair j
    const int src = __shfl_down_sync(0xffffffffu, here.slot, kPairs);
    if (lane < kPairs && i + lane < moved) {
      const float wv = __ldcg(w + src);
      const int32_t pv = __ldcg(pos + src);
      w[here.slot] = wv;
      w[src] = 0.f;
      pos[here.slot] = pv;
    }
    next = place_of(p, lists, r, i + step, moved, lane);
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      const int64_t dst = __shfl_sync(0xffffffffu, here.row, j);
      if (!from[j]) {
        if (lane == 0 && i + j < moved && p.err) atomicOr(p.err, SMLA_DEVERR_PAGE_RANGE);
        continue;
      }
      unsigned char* to = p.kv + dst * kRecordBytes;
      reinterpret_cast<uint4*>(to)[lane] = a[j];
      if (lane < kUnits - 32) reinterpret_cast<uint4*>(to)[32 + lane] = b[j];
    }
  }
}

cudaLaunchConfig_t select_config(int requests, int csize, cudaStream_t stream, cudaLaunchAttribute* a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)requests * csize);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kDynBytes;
  cfg.stream = stream;
  a->id = cudaLaunchAttributeClusterDimension;
  a->val.clusterDim.x = csize;
  a->val.clusterDim.y = a->val.clusterDim.z = 1;
  cfg.attrs = a;
  cfg.numAttrs = 1;
  return cfg;
}

// Sets the selection up on the current device; the largest cluster of it that the device can hold.
cudaError_t largest_cluster(int* most) {
  cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kDynBytes);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  for (*most = kEvictMostCluster; *most > 1; *most /= 2) {
    cudaLaunchAttribute a;
    const cudaLaunchConfig_t cfg = select_config(1, *most, nullptr, &a);
    int clusters = 0;
    if (cudaOccupancyMaxActiveClusters(&clusters, evict_select_kernel, &cfg) == cudaSuccess && clusters > 0) break;
    (void)cudaGetLastError();                          // (an answer, not an error of the call)
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, int sms, cudaStream_t stream) {
  if (p.requests == 0) return cudaSuccess;
  static std::atomic<int> most_of[64];                 // the devices' largest clusters, 0: not looked up yet
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int most = dev < 64 ? most_of[dev].load(std::memory_order_relaxed) : 0;
  if (most == 0) {
    e = largest_cluster(&most);
    if (e != cudaSuccess) return e;
    if (dev < 64) most_of[dev].store(most, std::memory_order_relaxed);
  }
  const int csize = evict_cluster(p.requests, p.cols, sms, most);
  cudaLaunchAttribute a;
  const cudaLaunchConfig_t cfg = select_config(p.requests, csize, stream, &a);
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
