// What the kernels over whole cached contexts share: rings of shared-memory slots, bounded waits, q as two E4M3 terms and
// the tensor maps of the cache.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include "smla_device.cuh"
#include "smla_internal.h"
#include "smla_ptx.cuh"

namespace smla {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

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
  __device__ __forceinline__ void skip(int n) {
    slot += n;
    if (slot >= N) {
      slot -= N;
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

// After a wait that gave up: every copy that was armed has to land before the CTA leaves.  Nothing arms a slot
// again by then, so the slot's last phase is waited for.
__device__ void drain_copies(uint64_t* bar, const int* armed, int n, int lane) {
  int never = 0;
  for (int s = 0; s < n; ++s)
    if (armed[s] > 0) ptx::mbar_wait_warp(&bar[s], (uint32_t)(armed[s] - 1) & 1u, &never, lane, 100000000ull);
}

__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// A row of q as two E4M3 terms: 16 latent values per lane (bf16 pairs) -> hi + lo of them times 2^-x, x (the same in every
// lane) such that the row's largest lies in [2^7, 2^8).
__device__ __forceinline__ int split_q(const uint32_t (&wds)[8], uint32_t (&hi)[4], uint32_t (&lo)[4]) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(wds[i] << 16)), fabsf(__uint_as_float(wds[i] & 0xffff0000u))));
#pragma unroll
  for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  // x = floor(log2 amax) - 7, kept where 2^x and 2^-x are normal floats
  const int x = amax > 0.f ? min(max((int)(__float_as_uint(amax) >> 23) - 127 - 7, -120), 120) : 0;
  const float down = exp2_int(-x);
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
  return x;
}

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiled encoder() {
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
inline bool encode_map(CUtensorMap* map, const uint8_t* kv, int64_t num_pages, uint32_t bytes, CUtensorMapSwizzle swizzle) {
  const cuuint64_t dims[3] = {kRecordBytes, kPageSize, (cuuint64_t)num_pages};
  const cuuint64_t strides[2] = {kRecordBytes, (cuuint64_t)kRecordBytes * kPageSize};
  const cuuint32_t box[3] = {bytes, kPageSize, 1}, step[3] = {1, 1, 1};
  return encoder()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(kv), dims, strides, box, step,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace smla
