// Reading records of the paged FP8 cache back: out[i] = [e4m3(code) * scale | rope], one token per warp.
// Bound by HBM bytes (656 read, 576 elements written per token).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "smla_device.cuh"
#include "smla_internal.h"

namespace smla {
namespace {

constexpr int kReadWarps = 8;

// fp32 pair -> two elements of the output type in one 32-bit word.
template <int kDtype>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (kDtype == SMLA_BF16) return f32x2_to_bf16x2(a, b);
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int kDtype>
__global__ void __launch_bounds__(32 * kReadWarps) kv_read_kernel(const ReadParams p) {
  const int lane = threadIdx.x & 31;
  const int tok = blockIdx.x * kReadWarps + (threadIdx.x >> 5);
  if (tok >= p.tokens) return;
  constexpr int kEsz = kDtype == SMLA_FP32 ? 4 : 2;
  unsigned char* out = static_cast<unsigned char*>(p.out) + (size_t)tok * kDQK * kEsz;
  const int req = p.requests ? __ldg(p.requests + tok) : tok;
  const int pos = __ldg(p.positions + tok);
  int page = -1;
  if (req >= 0 && req < p.num_requests && pos >= 0 && (pos >> 6) < p.max_pages)
    page = __ldg(p.block_table + (size_t)req * p.max_pages + (pos >> 6));
  uint4 codes = make_uint4(0u, 0u, 0u, 0u);
  float scale = 0.f;
  uint32_t rope = 0u;
  if (page < 0 || (int64_t)page >= p.num_pages) {
    if (lane == 0 && p.err) atomicOr(p.err, SMLA_DEVERR_PAGE_RANGE);
  } else {
    const unsigned char* rec = p.kv + ((int64_t)page * kPageSize + (pos & (kPageSize - 1))) * kRecordBytes;
    codes = __ldg(reinterpret_cast<const uint4*>(rec) + lane);
    scale = __ldg(reinterpret_cast<const float*>(rec + kDLatent) + (lane >> 3));
    rope = __ldg(reinterpret_cast<const uint32_t*>(rec + kDLatent + 16) + lane);
  }
  float v[16];
  const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = f16x2_to_f32x2(e4m3x2_to_f16x2((uint16_t)(w[i] & 0xffffu)));
    const float2 b = f16x2_to_f32x2(e4m3x2_to_f16x2((uint16_t)(w[i] >> 16)));
    v[4 * i] = a.x * scale;
    v[4 * i + 1] = a.y * scale;
    v[4 * i + 2] = b.x * scale;
    v[4 * i + 3] = b.y * scale;
  }
  const float r0 = __uint_as_float(rope << 16), r1 = __uint_as_float(rope & 0xFFFF0000u);
  if constexpr (kDtype == SMLA_FP32) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      reinterpret_cast<float4*>(out)[4 * lane + i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    reinterpret_cast<float2*>(out + kDLatent * 4)[lane] = make_float2(r0, r1);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      reinterpret_cast<uint4*>(out)[2 * lane + i] =
          make_uint4(pack2<kDtype>(v[8 * i], v[8 * i + 1]), pack2<kDtype>(v[8 * i + 2], v[8 * i + 3]),
                     pack2<kDtype>(v[8 * i + 4], v[8 * i + 5]), pack2<kDtype>(v[8 * i + 6], v[8 * i + 7]));
    // a bf16 rope goes out as it is stored (NaN payloads included)
    reinterpret_cast<uint32_t*>(out + kDLatent * 2)[lane] = kDtype == SMLA_BF16 ? rope : pack2<kDtype>(r0, r1);
  }
}

}  // namespace

cudaError_t launch_kv_read(const ReadParams& p, cudaStream_t stream) {
  if (p.tokens == 0) return cudaSuccess;
  const int blocks = (p.tokens + kReadWarps - 1) / kReadWarps;
  if (p.out_dtype == SMLA_BF16) kv_read_kernel<SMLA_BF16><<<blocks, 32 * kReadWarps, 0, stream>>>(p);
  else if (p.out_dtype == SMLA_FP16) kv_read_kernel<SMLA_FP16><<<blocks, 32 * kReadWarps, 0, stream>>>(p);
  else kv_read_kernel<SMLA_FP32><<<blocks, 32 * kReadWarps, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace smla
