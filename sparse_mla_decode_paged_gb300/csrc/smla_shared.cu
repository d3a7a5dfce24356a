// Decode of requests behind shared prefixes: every request attends over the positions of its group's prefix, then over its
// own, and the records of a prefix are read for all of the group's rows at once.
//
// The dense decode's kernel takes both kinds of items on one line of tiles (a prefix's rows are those of all its requests)
// and leaves two results per row in fp32; the join here makes one of them:
//   lse = ln(exp(lse_own) + exp(lse_prefix)), out = exp(lse_own - lse) out_own + exp(lse_prefix - lse) out_prefix.
#include <cuda_runtime.h>
#include <math_constants.h>

#include "smla_device.cuh"
#include "smla_internal.h"
#include "smla_ptx.cuh"

namespace smla {
namespace {

constexpr int kJoinThreads = 128;

// One warp per row, 16 dims per lane.  (This grid is resident while results are still written, so they are read from L2.)
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const float* o, const float* lse, uint16_t* out, float* lse_out,
                                                            int rows) {
  const int row = blockIdx.x * (kJoinThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  ptx::griddep_wait();
  if (row >= rows) return;
  const float4 *a = reinterpret_cast<const float4*>(o + (size_t)row * kDLatent),
               *b = reinterpret_cast<const float4*>(o + ((size_t)rows + row) * kDLatent);
  float4 x[4], y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = __ldcg(a + 32 * i + lane);
    y[i] = __ldcg(b + 32 * i + lane);
  }
  const float la = __ldcg(lse + row), lb = __ldcg(lse + rows + row);
  float m = fmaxf(la, lb);
  if (isnan(la) || isnan(lb)) m = CUDART_NAN_F;
  const float ea = m == -CUDART_INF_F ? 0.f : expf(la - m), eb = m == -CUDART_INF_F ? 0.f : expf(lb - m), z = ea + eb;
  const float wa = z == 0.f ? 0.f : ea / z, wb = z == 0.f ? 0.f : eb / z;
  uint2* to = reinterpret_cast<uint2*>(out + (size_t)row * kDLatent);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    to[32 * i + lane] = make_uint2(f32x2_to_bf16x2(fmaf(wa, x[i].x, wb * y[i].x), fmaf(wa, x[i].y, wb * y[i].y)),
                                   f32x2_to_bf16x2(fmaf(wa, x[i].z, wb * y[i].z), fmaf(wa, x[i].w, wb * y[i].w)));
  if (lane == 0) lse_out[row] = z == 0.f ? -CUDART_INF_F : m + logf(z);
}

}  // namespace

cudaError_t launch_shared(const SharedParams& p, cudaStream_t stream) {
  cudaError_t e = launch_dense(p.dense, stream);
  if (e != cudaSuccess) return e;
  const int rows = p.dense.B * p.dense.H;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((rows + kJoinThreads / 32 - 1) / (kJoinThreads / 32));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = a;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel, (const float*)p.dense.out32, (const float*)p.dense.lse32, p.out, p.lse, rows);
}

}  // namespace smla
