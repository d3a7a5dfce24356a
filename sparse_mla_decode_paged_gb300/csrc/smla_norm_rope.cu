// Norm and rotation in one pass: the fused write side of the paged cache (RMS norm of the latent,
// rotation of the rope part, FP8 quantisation, record write) and the per-head norm + rotation of
// query or key heads.
//
//   n_d = x_d / sqrt(mean x^2 + eps) * w_d;  rotation of a pair (a, b): (a c - b s, a s + b c).
//
// Both are bound by HBM bytes (a few dozen operations per element): each row is read once into
// registers, every step is done there in fp32, and the result is rounded once and written once.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "smla_device.cuh"
#include "smla_internal.h"

namespace smla {
namespace {

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// N consecutive elements as floats: 16-byte accesses (N * sizeof(T) a multiple of 16, p aligned), or
// element by element.
template <int N, typename T>
__device__ __forceinline__ void load_vec(const T* p, float (&v)[N]) {
  constexpr int kPer = 16 / sizeof(T);
#pragma unroll
  for (int i = 0; i < N / kPer; ++i) {
    const uint4 raw = *reinterpret_cast<const uint4*>(p + i * kPer);
    const T* e = reinterpret_cast<const T*>(&raw);
#pragma unroll
    for (int j = 0; j < kPer; ++j) v[i * kPer + j] = to_f32<T>(e[j]);
  }
}
template <int N, typename T>
__device__ __forceinline__ void load_each(const T* p, float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = to_f32<T>(p[i]);
}
template <int N, typename T>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[N]) {
  constexpr int kPer = 16 / sizeof(T);
#pragma unroll
  for (int i = 0; i < N / kPer; ++i) {
    uint4 raw;
    T* e = reinterpret_cast<T*>(&raw);
#pragma unroll
    for (int j = 0; j < kPer; ++j) e[j] = from_f32<T>(v[i * kPer + j]);
    *reinterpret_cast<uint4*>(p + i * kPer) = raw;
  }
}

// N weights at `at` (fp32, or the type of x).
template <int N, typename T>
__device__ __forceinline__ void load_weight(const void* w, int at, int weight_dtype, float (&v)[N]) {
  if (weight_dtype == SMLA_FP32)
    load_each<N, float>(static_cast<const float*>(w) + at, v);
  else
    load_each<N, T>(static_cast<const T*>(w) + at, v);
}

// ---------------------------------------------------------------------------- norm + rotation + append

constexpr int kNormAppendWarps = 4;

// One warp per token.  Lane l holds latent dims 16 l .. 16 l + 15 (block l / 8 of 128 dims, so a block's
// amax is a reduction over 8 lanes) and rope dims 2 l, 2 l + 1; the codes go out as one 16-byte store per
// lane.  The weights stay in registers over the warp's tokens.
template <typename T, bool kWide>
__global__ void __launch_bounds__(32 * kNormAppendWarps) kv_norm_append_kernel(const NormAppendParams p) {
  const int lane = threadIdx.x & 31;
  const int warps = gridDim.x * kNormAppendWarps;
  float w[16];
  load_weight<16, T>(p.weight, 16 * lane, p.weight_dtype, w);
  for (int tok = blockIdx.x * kNormAppendWarps + (threadIdx.x >> 5); tok < p.tokens; tok += warps) {
    const int req = p.requests ? __ldg(p.requests + tok) : tok;
    const int pos = __ldg(p.positions + tok);
    float x[16];
    const T* row = static_cast<const T*>(p.latent) + (int64_t)tok * p.latent_stride + 16 * lane;
    if constexpr (kWide) load_vec<16, T>(row, x); else load_each<16, T>(row, x);
    const T* rr = static_cast<const T*>(p.rope) + (int64_t)tok * p.rope_stride + 2 * lane;
    float r0 = to_f32<T>(rr[0]), r1 = to_f32<T>(rr[1]);
    int page = -1;
    if (req >= 0 && req < p.num_requests && pos >= 0 && (pos >> 6) < p.max_pages && pos < p.max_positions)
      page = __ldg(p.block_table + (size_t)req * p.max_pages + (pos >> 6));
    if (page < 0 || (int64_t)page >= p.num_pages) {
      if (lane == 0 && p.err) atomicOr(p.err, SMLA_DEVERR_PAGE_RANGE);
      continue;                                      // warp-uniform
    }
    unsigned char* rec = p.kv + ((int64_t)page * kPageSize + (pos & (kPageSize - 1))) * kRecordBytes;
    const float* cs = p.cos_sin + (size_t)pos * kDRope;

    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float inv = rsqrtf(ss * (1.f / kDLatent) + p.eps);
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      x[i] = x[i] * inv * w[i];
      amax = fmaxf(amax, fabsf(x[i]));
    }
#pragma unroll
    for (int o = 4; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    // the quantisation of sparse_mla_kv_append: two correctly rounded fp32 divisions, then E4M3
    const float scale = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint16_t lo = f32x2_to_e4m3x2(__fdiv_rn(x[4 * i], scale), __fdiv_rn(x[4 * i + 1], scale));
      const uint16_t hi = f32x2_to_e4m3x2(__fdiv_rn(x[4 * i + 2], scale), __fdiv_rn(x[4 * i + 3], scale));
      c[i] = (uint32_t)lo | ((uint32_t)hi << 16);
    }
    reinterpret_cast<uint4*>(rec)[lane] = make_uint4(c[0], c[1], c[2], c[3]);
    if ((lane & 7) == 0) reinterpret_cast<float*>(rec + kDLatent)[lane >> 3] = scale;

    float y0, y1;
    if (p.interleaved) {                             // this lane's two dims are pair `lane`
      const float co = __ldg(cs + lane), si = __ldg(cs + 32 + lane);
      y0 = r0 * co - r1 * si;
      y1 = r0 * si + r1 * co;
    } else {                                         // partners of dims 2 l, 2 l + 1 sit 16 lanes away
      const float q0 = __shfl_xor_sync(0xffffffffu, r0, 16), q1 = __shfl_xor_sync(0xffffffffu, r1, 16);
      const int j = (2 * lane) & 31;
      const float2 co = __ldg(reinterpret_cast<const float2*>(cs + j));
      const float2 si = __ldg(reinterpret_cast<const float2*>(cs + 32 + j));
      y0 = lane < 16 ? r0 * co.x - q0 * si.x : q0 * si.x + r0 * co.x;
      y1 = lane < 16 ? r1 * co.y - q1 * si.y : q1 * si.y + r1 * co.y;
    }
    reinterpret_cast<uint32_t*>(rec + kDLatent + 16)[lane] = f32x2_to_bf16x2(y0, y1);
  }
}

// ---------------------------------------------------------------------------- per-head norm + rotation

constexpr int kNormRopeThreads = 256;

// The rotated value of element e (of rotated dims o = e - rope_offset) from its own value v and its
// partner's value u.
__device__ __forceinline__ float rotated(const NormRopeParams& p, const float* cs, int o, float v, float u) {
  const int half = p.rope_dim >> 1;
  const int j = p.interleaved ? o >> 1 : (o < half ? o : o - half);
  const bool first = p.interleaved ? (o & 1) == 0 : o < half;
  const float c = __ldg(cs + j), s = __ldg(cs + half + j);
  return first ? v * c - u * s : u * s + v * c;
}

// One warp per (token, head) row, lane l holding elements l, l + 32, ...: any dim, stride and alignment.
template <typename T>
__global__ void __launch_bounds__(kNormRopeThreads) norm_rope_any_kernel(const NormRopeParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t rows = (int64_t)p.tokens * p.heads;
  const int64_t warps = (int64_t)gridDim.x * (kNormRopeThreads / 32);
  for (int64_t r = (int64_t)blockIdx.x * (kNormRopeThreads / 32) + (threadIdx.x >> 5); r < rows; r += warps) {
    const int t = (int)(r / p.heads), h = (int)(r % p.heads);
    const T* x = static_cast<const T*>(p.x) + (int64_t)t * p.x_token + (int64_t)h * p.x_head;
    T* out = static_cast<T*>(p.out) + (int64_t)t * p.out_token + (int64_t)h * p.out_head;
    int pos = 0;
    if (p.rope_dim) pos = __ldg(p.positions + t);
    if (p.rope_dim && (pos < 0 || pos >= p.max_positions)) {
      if (lane == 0 && p.err) atomicOr(p.err, SMLA_DEVERR_LEN_RANGE);
      for (int e = lane; e < p.dim; e += 32) out[e] = from_f32<T>(0.f);
      continue;
    }
    float v[kMaxNormRopeDim / 32];
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < kMaxNormRopeDim / 32; ++k) {
      const int e = lane + 32 * k;
      v[k] = e < p.dim ? to_f32<T>(x[e]) : 0.f;
      ss = fmaf(v[k], v[k], ss);
    }
    float inv = 1.f;
    if (p.norm) {
#pragma unroll
      for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      inv = rsqrtf(ss / (float)p.dim + p.eps);
    }
    auto weight = [&](int e) {
      if (!p.norm || !p.weight) return 1.f;
      return p.weight_dtype == SMLA_FP32 ? static_cast<const float*>(p.weight)[e]
                                         : to_f32<T>(static_cast<const T*>(p.weight)[e]);
    };
    const float* cs = p.cos_sin + (size_t)pos * p.rope_dim;
    const int half = p.rope_dim >> 1;
#pragma unroll
    for (int k = 0; k < kMaxNormRopeDim / 32; ++k) {
      const int e = lane + 32 * k, o = e - p.rope_offset;
      if (e >= p.dim) continue;
      v[k] = v[k] * inv * weight(e);
      if (o >= 0 && o < p.rope_dim) {
        const int pe = p.interleaved ? p.rope_offset + (o ^ 1) : (o < half ? e + half : e - half);
        v[k] = rotated(p, cs, o, v[k], to_f32<T>(x[pe]) * inv * weight(pe));
      }
    }
    __syncwarp();                                    // in place: every lane has read its partners
#pragma unroll
    for (int k = 0; k < kMaxNormRopeDim / 32; ++k) {
      const int e = lane + 32 * k;
      if (e < p.dim) out[e] = from_f32<T>(v[k]);
    }
  }
}

}  // namespace

cudaError_t launch_kv_norm_append(const NormAppendParams& p, cudaStream_t stream) {
  if (p.tokens == 0) return cudaSuccess;
  const int esz = p.dtype == SMLA_FP32 ? 4 : 2;
  const bool wide = reinterpret_cast<uintptr_t>(p.latent) % 16 == 0 && (p.latent_stride * esz) % 16 == 0;
  const int blocks = (p.tokens + kNormAppendWarps - 1) / kNormAppendWarps;
  auto go = [&](auto kernel) { kernel<<<blocks, 32 * kNormAppendWarps, 0, stream>>>(p); };
  if (p.dtype == SMLA_BF16)
    wide ? go(kv_norm_append_kernel<__nv_bfloat16, true>) : go(kv_norm_append_kernel<__nv_bfloat16, false>);
  else if (p.dtype == SMLA_FP16)
    wide ? go(kv_norm_append_kernel<__half, true>) : go(kv_norm_append_kernel<__half, false>);
  else
    wide ? go(kv_norm_append_kernel<float, true>) : go(kv_norm_append_kernel<float, false>);
  return cudaGetLastError();
}

cudaError_t launch_norm_rope(const NormRopeParams& p, cudaStream_t stream) {
  const int64_t rows = (int64_t)p.tokens * p.heads;
  if (rows == 0) return cudaSuccess;
  const int64_t want = (rows + kNormRopeThreads / 32 - 1) / (kNormRopeThreads / 32);
  const int blocks = (int)(want < (1 << 20) ? want : (1 << 20));
  auto go = [&](auto kernel) { kernel<<<blocks, kNormRopeThreads, 0, stream>>>(p); };
  if (p.dtype == SMLA_BF16) go(norm_rope_any_kernel<__nv_bfloat16>);
  else if (p.dtype == SMLA_FP16) go(norm_rope_any_kernel<__half>);
  else go(norm_rope_any_kernel<float>);
  return cudaGetLastError();
}

}  // namespace smla
