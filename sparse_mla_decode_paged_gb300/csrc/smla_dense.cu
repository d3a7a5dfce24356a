// Dense decode attention over the paged FP8 latent cache: every cached position of a request attends
// (no top-k list).  s_t = sm_scale q.k_t, out = softmax(s).v, lse = ln sum exp(s); each record is
// k = [e4m3(code) * scale | rope], v = k[0..511].
//
// One CTA per (query, head): its 8 warps walk the positions in turn, each with a running maximum and
// sum, and merge at the end.
#include <cuda_runtime.h>
#include <math_constants.h>

#include "smla_device.cuh"
#include "smla_internal.h"
#include "smla_ptx.cuh"

namespace smla {
namespace {

constexpr int kWarps = 8;

__global__ void __launch_bounds__(32 * kWarps) dense_kernel(const DenseParams p) {
  const int row = blockIdx.x, b = row / p.H;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t table_len = (int64_t)p.max_pages * kPageSize;
  int len = max(__ldg(p.seq_lens + b), 0);
  if (len > table_len) {
    if (threadIdx.x == 0) atomicOr(p.err, SMLA_DEVERR_PAGE_RANGE);
    len = (int)table_len;
  }
  const int32_t* bt = p.block_table + (size_t)(b / p.q_per_req) * p.max_pages;
  const uint16_t* q = p.q + (size_t)row * kDQK;
  float ql[16], qr[2];
  for (int i = 0; i < 16; ++i) ql[i] = bf16_to_f32(q[16 * lane + i]);
  for (int i = 0; i < 2; ++i) qr[i] = bf16_to_f32(q[kDLatent + 2 * lane + i]);
  float m = -CUDART_INF_F, l = 0.f, acc[16] = {};
  for (int t = warp; t < len; t += kWarps) {
    const int64_t r = row_of(bt, t, len, p.max_pages, p.num_pages, p.err);
    if (r < 0) continue;
    const unsigned char* rec = p.kv + r * kRecordBytes;
    const uint4 codes = __ldg(reinterpret_cast<const uint4*>(rec) + lane);
    const float scale = __ldg(reinterpret_cast<const float*>(rec + kDLatent) + (lane >> 3));
    const uint32_t rope = __ldg(reinterpret_cast<const uint32_t*>(rec + kDLatent + 16) + lane);
    const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
    float v[16], s = 0.f;
    for (int i = 0; i < 4; ++i) {
      const float2 a = f16x2_to_f32x2(e4m3x2_to_f16x2((uint16_t)(w[i] & 0xffffu)));
      const float2 c = f16x2_to_f32x2(e4m3x2_to_f16x2((uint16_t)(w[i] >> 16)));
      v[4 * i] = a.x * scale;
      v[4 * i + 1] = a.y * scale;
      v[4 * i + 2] = c.x * scale;
      v[4 * i + 3] = c.y * scale;
    }
    bool over = false;
    for (int i = 0; i < 16; ++i) {
      over |= fabsf(v[i]) > 65504.f;
      s = fmaf(ql[i], v[i], s);
    }
    if (over) atomicOr(p.err, SMLA_DEVERR_RANGE);
    s = fmaf(qr[0], __uint_as_float(rope << 16), s);
    s = fmaf(qr[1], __uint_as_float(rope & 0xFFFF0000u), s);
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    s *= p.sm_scale;
    if (isnan(s)) m = s;                             // the row's result is NaN
    const float mn = fmaxf(m, s), c = m == -CUDART_INF_F ? 0.f : expf(m - mn), e = expf(s - mn);
    l = l * c + e;
    for (int i = 0; i < 16; ++i) acc[i] = acc[i] * c + e * v[i];
    if (!isnan(m)) m = mn;
  }
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][kDLatent];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  for (int i = 0; i < 16; ++i) so[warp][16 * lane + i] = acc[i];
  __syncthreads();
  float mx = -CUDART_INF_F, z = 0.f;
  for (int w = 0; w < kWarps; ++w) mx = isnan(sm[w]) || isnan(mx) ? CUDART_NAN_F : fmaxf(mx, sm[w]);
  for (int w = 0; w < kWarps; ++w) z += sm[w] == -CUDART_INF_F ? 0.f : sl[w] * expf(sm[w] - mx);
  const float inv = z > 0.f ? 1.f / z : (z == 0.f ? 0.f : CUDART_NAN_F);
  for (int d = 2 * threadIdx.x; d < kDLatent; d += 2 * 32 * kWarps) {
    float o0 = 0.f, o1 = 0.f;
    for (int w = 0; w < kWarps; ++w) {
      const float c = sm[w] == -CUDART_INF_F ? 0.f : expf(sm[w] - mx);
      o0 += c * so[w][d];
      o1 += c * so[w][d + 1];
    }
    reinterpret_cast<uint32_t*>(p.out + (size_t)row * kDLatent)[d / 2] = f32x2_to_bf16x2(o0 * inv, o1 * inv);
  }
  if (threadIdx.x == 0) p.lse[row] = z == 0.f ? -CUDART_INF_F : mx + logf(z);
}

}  // namespace

cudaError_t launch_dense(const DenseParams& p, cudaStream_t stream) {
  dense_kernel<<<p.B * p.H, 32 * kWarps, 0, stream>>>(p);
  return cudaGetLastError();
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
  plan->rows_per_cta = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
  plan->row_groups = (int32_t)((rows + plan->rows_per_cta - 1) / plan->rows_per_cta);
  plan->ctas = d->ctas > 0 ? d->ctas : (sm_count < kDenseMaxCtas ? sm_count : kDenseMaxCtas);
  plan->reserved = 0;
  plan->workspace_bytes = kWorkspaceHeader;
  return SMLA_OK;
}
