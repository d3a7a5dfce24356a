// Decode of requests behind shared prefixes: every request attends over the positions of its group's prefix, then over its
// own, and the records of a prefix are read for all of the group's rows at once.
//
// Short prefixes and few rows: the dense decode's kernel takes both kinds of items on one line of tiles (a prefix's rows
// are those of all its requests).  Else the prefix kernel takes the prefixes and, where they are short, the requests' own
// positions, too; long ones stay with the dense kernel.  Either way results per row are left in fp32, and the join here makes one of them:
//   lse = ln sum_i exp(lse_i), out = sum_i exp(lse_i - lse) out_i.
#include <cuda_runtime.h>
#include <math_constants.h>

#include "smla_device.cuh"
#include "smla_internal.h"
#include "smla_prefix_parts.cuh"
#include "smla_ptx.cuh"

namespace smla {
namespace {

constexpr int kJoinDims = 128;             // threads that share a row's 512 dims
constexpr int kJoinGroups = 4;            // groups of them that share its parts, where they are many
constexpr int kJoinBatch = 8;             // parts in flight per thread
constexpr int kManyParts = 24;
constexpr int kMostParts = 2 * kDenseMaxCtas;

// Where a row's results lie: `parts` of them, the s-th at place(s) of the arrays.
struct Parts {
  const float *o, *lse;
  int parts, pair, at, rows;              // one result at row `at`, or parts in slots of `rows` rows from that pair (or CTA) on
  __device__ __forceinline__ size_t place(int s) const {
    return parts == 1 ? (size_t)at : (size_t)(2 * (pair + s) + (s == 0 ? 1 : 0)) * rows + at;
  }
};

// The dense kernel's side of a call.
struct DenseItems {
  DenseSlots slots;
  int ctas, nr, groups, prefix_groups;    // rows per slot, row groups per request and per prefix
};

// The prefix kernel's results of row r of segment g: a whole one lies with the rows, the first of several in slot 1 of its
// pair, the others in slot 0 of theirs.
__device__ __forceinline__ Parts segment_parts(const PrefixParams& p, int g, int row) {
  const Segment seg = segment_of(p, g);
  const int r = row - seg.first_row, block = r / kPrefixRows;
  Parts x{p.slots, p.slots_lse, 0, 0, r - block * kPrefixRows, kPrefixRows};
  const long long* ends = p.begins + segments_of(p);
  const long long total = __ldcg(ends), start = __ldcg(ends + 1), begin = __ldcg(p.begins + g);
  const long long units = (__ldcg(p.begins + g + 1) - begin) / seg.blocks;       // of an item
  if (units == 0) return x;
  const long long a = begin + block * units + start, e = begin + (block + 1) * units;
  const int active = active_pairs(total, p.pairs);
  auto about = [&](long long u) {                          // the pair whose run holds unit u, give or take one
    const unsigned long long x = (unsigned long long)u * active;
    return (int)min((unsigned long long)active - 1,
                    (x | (unsigned long long)total) >> 32 ? x / total : (uint32_t)x / (uint32_t)total);
  };
  int c = about(a);
  while (c > 0 && pair_start(total, active, c) > a) --c;
  while (c + 1 < active && pair_start(total, active, c + 1) <= a) ++c;
  int c1 = max(c, about(e));
  while (c1 > c && pair_start(total, active, c1) >= e) --c1;
  while (c1 + 1 < active && pair_start(total, active, c1 + 1) < e) ++c1;
  x.parts = c1 - c + 1;
  x.pair = c;
  if (x.parts == 1) {
    x.o = p.out32 + (seg.own ? 0 : p.all_rows) * kDLatent;
    x.lse = p.lse32 + (seg.own ? 0 : p.all_rows);
    x.at = row;
  }
  return x;
}

// Joins a row's parts, those of a before those of b.  A group of 128 threads takes 4 dims each of every kGroups-th part.
template <int kGroups>
__device__ __forceinline__ void join_row(const Parts& a, const Parts& b, uint16_t* out, float* lse_out, int row) {
  __shared__ float w_s[kMostParts], z_s;
  __shared__ float4 sum_s[kGroups][kJoinDims];
  const int lane = threadIdx.x & 31, dim = threadIdx.x % kJoinDims, group = threadIdx.x / kJoinDims;
  const int parts = a.parts + b.parts;
  auto row_of = [&](int s) {
    return reinterpret_cast<const float4*>(s < a.parts ? a.o + a.place(s) * kDLatent : b.o + b.place(s - a.parts) * kDLatent) + dim;
  };
  float4 v[kJoinBatch];                                    // in flight before the weights are known
#pragma unroll
  for (int j = 0; j < kJoinBatch; ++j)
    if (group + kGroups * j < parts) v[j] = __ldcg(row_of(group + kGroups * j));
  if (threadIdx.x < 32) {
    float m = -CUDART_INF_F;
    bool bad = false;
    for (int s = lane; s < parts; s += 32) {
      const float x = __ldcg(s < a.parts ? a.lse + a.place(s) : b.lse + b.place(s - a.parts));
      w_s[s] = x;
      bad |= isnan(x);
      m = fmaxf(m, x);
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
    if (lane == 0) {
      z_s = z;
      lse_out[row] = z == 0.f ? -CUDART_INF_F : m + logf(z);
    }
  }
  __syncthreads();
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = group; s0 < parts; s0 += kGroups * kJoinBatch) {
    if (s0 > group) {
#pragma unroll
      for (int j = 0; j < kJoinBatch; ++j)
        if (s0 + kGroups * j < parts) v[j] = __ldcg(row_of(s0 + kGroups * j));
    }
#pragma unroll
    for (int j = 0; j < kJoinBatch; ++j) {
      if (s0 + kGroups * j >= parts) continue;
      const float w = w_s[s0 + kGroups * j];
      acc.x = fmaf(w, v[j].x, acc.x);
      acc.y = fmaf(w, v[j].y, acc.y);
      acc.z = fmaf(w, v[j].z, acc.z);
      acc.w = fmaf(w, v[j].w, acc.w);
    }
  }
  if constexpr (kGroups > 1) {
    sum_s[group][dim] = acc;
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int i = 1; i < kGroups; ++i) {
      const float4 x = sum_s[i][dim];
      acc.x += x.x;
      acc.y += x.y;
      acc.z += x.z;
      acc.w += x.w;
    }
  }
  const float inv = z_s == 0.f ? 0.f : 1.f / z_s;
  reinterpret_cast<uint2*>(out + (size_t)row * kDLatent)[dim] =
      make_uint2(f32x2_to_bf16x2(acc.x * inv, acc.y * inv), f32x2_to_bf16x2(acc.z * inv, acc.w * inv));
}

// One CTA per row.  (This grid is resident while results are still written, so they are read from L2.)
template <int kGroups>
__global__ void __launch_bounds__(kJoinDims * kGroups) join_kernel(const PrefixParams p, const DenseItems d, uint16_t* out,
                                                                   float* lse_out) {
  __shared__ Parts own_s, prefix_s;
  const int row = blockIdx.x;
  const int own_rows = p.q_per_req * p.H, req = row / own_rows, prefix = row / p.rows;
  const bool own_dense = !p.own, prefix_dense = p.pairs == 0;
  // the dense kernel's items of this row, and its row in them
  const int own_group = own_dense ? (row - req * own_rows) / d.nr : 0;
  const int prefix_group = prefix_dense ? (row - prefix * p.rows) / d.nr : 0;
  if (threadIdx.x == 0 && own_dense) own_s = Parts{p.out32, p.lse32, 1, 0, row, 0};
  if (threadIdx.x == 0 && prefix_dense)
    prefix_s = Parts{p.out32 + p.all_rows * kDLatent, p.lse32 + p.all_rows, 1, 0, row, 0};
  __syncthreads();
  ptx::griddep_wait();
  if (threadIdx.x == 0 && !own_dense) own_s = segment_parts(p, p.prefixes + req, row);
  if (threadIdx.x == 32 && !prefix_dense) prefix_s = segment_parts(p, prefix, row);
  if (own_dense) {
    const int own_item = req * d.groups + own_group;
    const int prefix_item = prefix_dense ? p.requests * d.groups + prefix * d.prefix_groups + prefix_group : -1;
    for (int c = threadIdx.x; c < d.ctas; c += kJoinDims * kGroups) {
      const int2 x = __ldcg(d.slots.descs + c);            // {item, parts}; an item is found at most once
      if (x.y > 0 && x.x == own_item)
        own_s = Parts{d.slots.o, d.slots.lse, x.y, c, row - req * own_rows - own_group * d.nr, d.nr};
      if (x.y > 0 && x.x == prefix_item)
        prefix_s = Parts{d.slots.o, d.slots.lse, x.y, c, row - prefix * p.rows - prefix_group * d.nr, d.nr};
    }
  }
  __syncthreads();
  join_row<kGroups>(own_s, prefix_s, out, lse_out, row);
}

// The same for a call without prefixes: rows of items that cross runs alone, the others are written.
template <int kGroups>
__global__ void __launch_bounds__(kJoinDims * kGroups) row_merge_kernel(const DenseItems d, int item_rows, uint16_t* out,
                                                                        float* lse_out) {
  __shared__ Parts found_s;
  const int row = blockIdx.x, req = row / item_rows, in = row - req * item_rows, item = req * d.groups + in / d.nr;
  if (threadIdx.x == 0) found_s.parts = 0;
  __syncthreads();
  ptx::griddep_wait();
  for (int c = threadIdx.x; c < d.ctas; c += kJoinDims * kGroups) {
    const int2 x = __ldcg(d.slots.descs + c);              // {item, parts}; an item is found at most once
    if (x.y > 0 && x.x == item) found_s = Parts{d.slots.o, d.slots.lse, x.y, c, in % d.nr, d.nr};
  }
  __syncthreads();
  if (found_s.parts > 0) join_row<kGroups>(found_s, Parts{}, out, lse_out, row);
}

}  // namespace

namespace {
DenseItems items_of(const DenseParams& p) {
  DenseItems d{};
  d.slots = dense_slots(p);
  d.ctas = p.ctas;
  d.nr = p.nr;
  d.groups = p.groups;
  d.prefix_groups = p.prefix_groups;
  return d;
}

cudaLaunchConfig_t dependent(unsigned grid, unsigned block, cudaStream_t stream, cudaLaunchAttribute* a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.stream = stream;
  a->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a->val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = a;
  cfg.numAttrs = 1;
  return cfg;
}
}  // namespace

cudaError_t launch_row_merge(const DenseParams& p, cudaStream_t stream) {
  const bool many = p.ctas / ((long long)p.requests * p.groups) > kManyParts;
  cudaLaunchAttribute a;
  const cudaLaunchConfig_t cfg = dependent((unsigned)(p.B * p.H), many ? kJoinDims * kJoinGroups : kJoinDims, stream, &a);
  return many ? cudaLaunchKernelEx(&cfg, row_merge_kernel<kJoinGroups>, items_of(p), p.q_per_req * p.H, p.out, p.lse)
              : cudaLaunchKernelEx(&cfg, row_merge_kernel<1>, items_of(p), p.q_per_req * p.H, p.out, p.lse);
}

cudaError_t launch_shared(const SharedParams& p, cudaStream_t stream) {
  const PrefixParams& x = p.prefix;
  cudaError_t e = x.pairs > 0 ? launch_prefix(x, stream) : cudaSuccess;
  if (e != cudaSuccess) return e;
  if (!x.own) e = launch_dense(p.dense, stream);
  if (e != cudaSuccess) return e;
  const DenseItems d = x.own ? DenseItems{} : items_of(p.dense);
  // parts of a prefix's block of rows, about
  const long long parts = x.pairs > 0 ? x.pairs / ((long long)x.prefixes * x.row_blocks)
                                      : p.dense.ctas / ((long long)x.prefixes * p.dense.prefix_groups);
  cudaLaunchAttribute a;
  const cudaLaunchConfig_t cfg =
      dependent((unsigned)x.all_rows, parts > kManyParts ? kJoinDims * kJoinGroups : kJoinDims, stream, &a);
  return parts > kManyParts ? cudaLaunchKernelEx(&cfg, join_kernel<kJoinGroups>, x, d, p.out, p.lse)
                            : cudaLaunchKernelEx(&cfg, join_kernel<1>, x, d, p.out, p.lse);
}

}  // namespace smla
