// Reading records of the paged FP8 cache back: out[i] = [e4m3(code) * scale | rope].
// Bound by HBM bytes (656 read, 576 elements written per token).  Measured, 131071 records to bf16: 38.3 us (6.2 TB/s);
// 16 dims of one block per lane, whose accesses leave gaps, took 44 us.
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

// Two tokens per warp, their loads in flight together.  Lane l takes dims 8 l .. 8 l + 7 and 256 + 8 l .. (8 codes
// each), so that every access of the warp is contiguous, and rope dims 2 l, 2 l + 1.
constexpr int kReadTokens = 2;

template <int kDtype>
__global__ void __launch_bounds__(32 * kReadWarps) kv_read_kernel(const ReadParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t first = ((int64_t)blockIdx.x * kReadWarps + (threadIdx.x >> 5)) * kReadTokens;
  constexpr int kEsz = kDtype == SMLA_FP32 ? 4 : 2;
  const unsigned char* rec[kReadTokens];
#pragma unroll
  for (int n = 0; n < kReadTokens; ++n) {
    const int64_t tok = first + n;
    rec[n] = nullptr;
    if (tok >= p.tokens) continue;
    const int req = p.requests ? __ldg(p.requests + tok) : (int)tok;
    const int pos = __ldg(p.positions + tok);
    int page = -1;
    if (req >= 0 && req < p.num_requests && pos >= 0 && (pos >> 6) < p.max_pages)
      page = __ldg(p.block_table + (size_t)req * p.max_pages + (pos >> 6));
    if (page >= 0 && (int64_t)page < p.num_pages)
      rec[n] = p.kv + ((int64_t)page * kPageSize + (pos & (kPageSize - 1))) * kRecordBytes;
    else if (lane == 0 && p.err)
      atomicOr(p.err, SMLA_DEVERR_PAGE_RANGE);
  }
  uint2 codes[kReadTokens][2];
  float scale[kReadTokens][2];
  uint32_t rope[kReadTokens];
#pragma unroll
  for (int n = 0; n < kReadTokens; ++n) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      codes[n][h] = rec[n] ? __ldg(reinterpret_cast<const uint2*>(rec[n]) + 32 * h + lane) : make_uint2(0u, 0u);
      scale[n][h] = rec[n] ? __ldg(reinterpret_cast<const float*>(rec[n] + kDLatent) + 2 * h + (lane >> 4)) : 0.f;
    }
    rope[n] = rec[n] ? __ldg(reinterpret_cast<const uint32_t*>(rec[n] + kDLatent + 16) + lane) : 0u;
  }
#pragma unroll
  for (int n = 0; n < kReadTokens; ++n) {
    if (first + n >= p.tokens) break;
    unsigned char* out = static_cast<unsigned char*>(p.out) + (size_t)(first + n) * kDQK * kEsz;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t w[2] = {codes[n][h].x, codes[n][h].y};
      float v[8];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 a = f16x2_to_f32x2(e4m3x2_to_f16x2((uint16_t)(w[i] & 0xffffu)));
        const float2 b = f16x2_to_f32x2(e4m3x2_to_f16x2((uint16_t)(w[i] >> 16)));
        v[4 * i] = a.x * scale[n][h];
        v[4 * i + 1] = a.y * scale[n][h];
        v[4 * i + 2] = b.x * scale[n][h];
        v[4 * i + 3] = b.y * scale[n][h];
      }
      if constexpr (kDtype == SMLA_FP32) {
        float4* o = reinterpret_cast<float4*>(out) + 64 * h + 2 * lane;
        o[0] = make_float4(v[0], v[1], v[2], v[3]);
        o[1] = make_float4(v[4], v[5], v[6], v[7]);
      } else {
        reinterpret_cast<uint4*>(out)[32 * h + lane] = make_uint4(pack2<kDtype>(v[0], v[1]), pack2<kDtype>(v[2], v[3]),
                                                                 pack2<kDtype>(v[4], v[5]), pack2<kDtype>(v[6], v[7]));
      }
    }
    const float r0 = __uint_as_float(rope[n] << 16), r1 = __uint_as_float(rope[n] & 0xFFFF0000u);
    if constexpr (kDtype == SMLA_FP32)
      reinterpret_cast<float2*>(out + kDLatent * 4)[lane] = make_float2(r0, r1);
    else                     // a bf16 rope goes out as it is stored (NaN payloads included)
      reinterpret_cast<uint32_t*>(out + kDLatent * 2)[lane] = kDtype == SMLA_BF16 ? rope[n] : pack2<kDtype>(r0, r1);
  }
}

}  // namespace

cudaError_t launch_kv_read(const ReadParams& p, cudaStream_t stream) {
  if (p.tokens == 0) return cudaSuccess;
  const int blocks = (int)(((int64_t)p.tokens + kReadWarps * kReadTokens - 1) / (kReadWarps * kReadTokens));
  if (p.out_dtype == SMLA_BF16) kv_read_kernel<SMLA_BF16><<<blocks, 32 * kReadWarps, 0, stream>>>(p);
  else if (p.out_dtype == SMLA_FP16) kv_read_kernel<SMLA_FP16><<<blocks, 32 * kReadWarps, 0, stream>>>(p);
  else kv_read_kernel<SMLA_FP32><<<blocks, 32 * kReadWarps, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace smla
