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

// N consecutive elements as floats.
template <int N, typename T>
__device__ __forceinline__ void load_each(const T* p, float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = to_f32<T>(p[i]);
}
// And back, rounded, in 16-byte stores.
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

// ---------------------------------------------------------------------------- norm + rotation + append

// 8 weights at `at` (fp32, or the type of x), which stay in L1.
template <typename T, bool kWide>
__device__ __forceinline__ void load_weights(const void* w, int at, int weight_dtype, float (&v)[8]) {
  if (weight_dtype == SMLA_FP32) {
    const float* p = static_cast<const float*>(w) + at;
    if constexpr (kWide) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
      const float f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = f[i];
    } else {
      load_each<8, float>(p, v);
    }
  } else if constexpr (sizeof(T) == 2) {
    const T* p = static_cast<const T*>(w) + at;
    if constexpr (kWide) {
      const uint4 raw = __ldg(reinterpret_cast<const uint4*>(p));
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = to_f32<T>(reinterpret_cast<const T*>(&raw)[i]);
    } else {
      load_each<8, T>(p, v);
    }
  }
}

constexpr int kNormAppendWarps = 4;
// Resident at once.  65521 tokens / 32 tokens with 6 (80 registers) 27.7 / 2.79 us, with 7 (72) 26.6 / 2.95: the small call, a
// step's, weighs more; with 5 the large one takes 6 % longer.
constexpr int kNormAppendBlocksPerSm = 6;

// Half a warp per token (two tokens per warp).  Lane l of a half takes
// dims 8 l .. 8 l + 7 of each 128-dim block, so every access of the warp is contiguous and a block's amax is a
// reduction over the 16 lanes; the four reductions share their exchanges (each lane ends with one block's amax and
// forms that block's scale and reciprocal).  What bounds it: HBM bytes (1152 read, 256 of cos and sin mostly from L2, 656
// written per token of a 16-bit type) and, behind them, issue.  Measured, 65521 bf16 tokens: 27.5 us (4.3 TB/s of these
// bytes without the table); a warp per token, which repeats the addresses, divisions and reductions, 31 us; with the
// next token's loads in flight as well (half the warps) 34 us.
template <typename T, bool kWide>
__global__ void __launch_bounds__(32 * kNormAppendWarps, kNormAppendBlocksPerSm)
    kv_norm_append_kernel(const NormAppendParams p) {
  constexpr int kPer = 16 / sizeof(T);
  const int lane = threadIdx.x & 31, l = lane & 15, half = lane >> 4;
  const int64_t step = 2 * (int64_t)gridDim.x * kNormAppendWarps;
  for (int64_t t0 = 2 * ((int64_t)blockIdx.x * kNormAppendWarps + (threadIdx.x >> 5)); t0 < p.tokens; t0 += step) {
    const int64_t tok = t0 + half;
    const bool in = tok < p.tokens;
    alignas(16) T x[32], r[4];
    int pos = -1, page = -1;
    if (in) {
      const int req = p.requests ? __ldg(p.requests + tok) : (int)tok;
      pos = __ldg(p.positions + tok);
      const T* row = static_cast<const T*>(p.latent) + tok * p.latent_stride + 8 * l;
      const T* rr = static_cast<const T*>(p.rope) + tok * p.rope_stride + 4 * l;
      if constexpr (kWide) {
#pragma unroll
        for (int i = 0; i < 32; i += kPer)
          *reinterpret_cast<uint4*>(x + i) = *reinterpret_cast<const uint4*>(row + 128 * (i / 8) + i % 8);
        if constexpr (sizeof(T) == 4) *reinterpret_cast<uint4*>(r) = *reinterpret_cast<const uint4*>(rr);
        else *reinterpret_cast<uint2*>(r) = *reinterpret_cast<const uint2*>(rr);
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = row[128 * (i / 8) + i % 8];
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = rr[i];
      }
      if (req >= 0 && req < p.num_requests && pos >= 0 && (pos >> 6) < p.max_pages && pos < p.max_positions)
        page = __ldg(p.block_table + (size_t)req * p.max_pages + (pos >> 6));
      if (page < 0 || (int64_t)page >= p.num_pages) {
        if (l == 0 && p.err) atomicOr(p.err, SMLA_DEVERR_PAGE_RANGE);
        page = -1;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] = from_f32<T>(0.f);
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = from_f32<T>(0.f);
    }
    const bool write = page >= 0;
    unsigned char* rec = p.kv + (write ? ((int64_t)page * kPageSize + (pos & (kPageSize - 1))) * kRecordBytes : 0);
    const float* cs = p.cos_sin + (write ? (size_t)pos * kDRope : 0);

    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) ss = fmaf(to_f32<T>(x[i]), to_f32<T>(x[i]), ss);
#pragma unroll
    for (int o = 8; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float inv = __frsqrt_rn(ss * (1.f / kDLatent) + p.eps);
    float n[32], amax[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      float f[8];
      load_weights<T, kWide>(p.weight, 128 * b + 8 * l, p.weight_dtype, f);
      amax[b] = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        n[8 * b + i] = to_f32<T>(x[8 * b + i]) * inv * f[i];
        amax[b] = fmaxf(amax[b], fabsf(n[8 * b + i]));
      }
    }
    // lane l ends with block 2 (l / 8) + (l / 4) % 2
    const bool hi8 = l & 8, hi4 = l & 4;
    float m0 = fmaxf(hi8 ? amax[2] : amax[0], __shfl_xor_sync(0xffffffffu, hi8 ? amax[0] : amax[2], 8));
    float m1 = fmaxf(hi8 ? amax[3] : amax[1], __shfl_xor_sync(0xffffffffu, hi8 ? amax[1] : amax[3], 8));
    float m = fmaxf(hi4 ? m1 : m0, __shfl_xor_sync(0xffffffffu, hi4 ? m0 : m1, 4));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    float scale = m > 0.f ? __fdiv_rn(m, 448.f) : 1.f;
    if (scale == 0.f) scale = 1.f;                   // amax below the smallest float's 224 fold: codes of 0
    const bool tiny = scale < 0x1p-100f;             // its reciprocal may not be a float: both sides times 2^64
    const float div = tiny ? scale * 0x1p64f : scale;
    const float up = __frcp_rn(div);
    const bool any_tiny = __any_sync(0xffffffffu, tiny);
    if (write && (l & 3) == 0) reinterpret_cast<float*>(rec + kDLatent)[l >> 2] = scale;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int from = 16 * half + 4 * b;
      const float u = __shfl_sync(0xffffffffu, up, from), d = -__shfl_sync(0xffffffffu, div, from);
      float* v = n + 8 * b;
      if (__builtin_expect(any_tiny, 0)) {
        const float lift = __shfl_sync(0xffffffffu, tiny ? 0x1p64f : 1.f, from);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= lift;
      }
      // n / scale: the product with the reciprocal, corrected once by its remainder (Markstein's division step), so that
      // the codes are those of the quotient rounded to fp32
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float q = v[i] * u;
        v[i] = fmaf(fmaf(q, d, v[i]), u, q);
      }
      uint32_t c[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        c[i] = (uint32_t)f32x2_to_e4m3x2(v[4 * i], v[4 * i + 1]) |
               ((uint32_t)f32x2_to_e4m3x2(v[4 * i + 2], v[4 * i + 3]) << 16);
      if (write) reinterpret_cast<uint2*>(rec)[16 * b + l] = make_uint2(c[0], c[1]);
    }

    // rope dims 4 l .. 4 l + 3
    float v[4], y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = to_f32<T>(r[i]);
    if (p.interleaved) {                             // pairs 2 l and 2 l + 1
      const float2 co = __ldg(reinterpret_cast<const float2*>(cs) + l);
      const float2 si = __ldg(reinterpret_cast<const float2*>(cs + 32) + l);
      y[0] = v[0] * co.x - v[1] * si.x;
      y[1] = v[0] * si.x + v[1] * co.x;
      y[2] = v[2] * co.y - v[3] * si.y;
      y[3] = v[2] * si.y + v[3] * co.y;
    } else {                                         // partners 32 dims, or 8 lanes, away
      const float4 co = __ldg(reinterpret_cast<const float4*>(cs) + (l & 7));
      const float4 si = __ldg(reinterpret_cast<const float4*>(cs + 32) + (l & 7));
      const float c4[4] = {co.x, co.y, co.z, co.w}, s4[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float q = __shfl_xor_sync(0xffffffffu, v[i], 8);
        y[i] = l < 8 ? v[i] * c4[i] - q * s4[i] : q * s4[i] + v[i] * c4[i];
      }
    }
    if (write)
      reinterpret_cast<uint2*>(rec + kDLatent + 16)[l] = make_uint2(f32x2_to_bf16x2(y[0], y[1]), f32x2_to_bf16x2(y[2], y[3]));
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

// A 16-byte unit as floats, and back.
template <typename T>
__device__ __forceinline__ void unpack(const uint4& raw, float (&v)[16 / sizeof(T)]) {
  const T* e = reinterpret_cast<const T*>(&raw);
#pragma unroll
  for (int i = 0; i < (int)(16 / sizeof(T)); ++i) v[i] = to_f32<T>(e[i]);
}

// N consecutive floats of a table row (aligned to N * 4 bytes, at most 16).
template <int N>
__device__ __forceinline__ void load_table(const float* p, float (&v)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 f = __ldg(reinterpret_cast<const float4*>(p + i));
      v[i] = f.x;
      v[i + 1] = f.y;
      v[i + 2] = f.z;
      v[i + 3] = f.w;
    }
  } else {
    const float2 f = __ldg(reinterpret_cast<const float2*>(p));
    v[0] = f.x;
    v[1] = f.y;
  }
}

// Whole 16-byte units (E elements): kLanes lanes per row, kUnits units per lane (unit u = lane + kLanes i), 32 / kLanes
// rows per warp at once.  A row stays in registers as it was loaded and is widened unit by unit, and so do a lane's
// weights over its rows, so that enough warps fit an SM to keep HBM busy (as floats: 102 us for 8192 x 64 x 192 in
// bf16, in units: 73 us).  What bounds it: HBM bytes (each element read once and written once; the rows of cos and sin
// stay in L1 over a token's heads).
template <typename T, int kLanes, int kUnits, bool kInterleaved>
__global__ void __launch_bounds__(kNormRopeThreads) norm_rope_kernel(const NormRopeParams p) {
  constexpr int E = 16 / sizeof(T), kRows = 32 / kLanes;
  const int lane = threadIdx.x & (kLanes - 1);
  const int units = p.dim / E, half = p.rope_dim >> 1;
  const uint32_t rows = (uint32_t)p.tokens * (uint32_t)p.heads;
  const uint32_t step = gridDim.x * (kNormRopeThreads / kLanes);
  const bool weighted = p.norm && p.weight;
  const bool narrow = weighted && p.weight_dtype == p.dtype;
  // the weights of unit u: kept where they have x's type, read again (from L1) where they are wider
  uint4 wraw[kUnits];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int u = lane + kLanes * i;
    wraw[i] = narrow && u < units ? __ldg(static_cast<const uint4*>(p.weight) + u) : make_uint4(0u, 0u, 0u, 0u);
  }
  auto scaled = [&](const uint4& raw, const uint4& w, int u, float inv, float (&v)[E]) {
    unpack<T>(raw, v);
    float f[E];
    if (narrow) unpack<T>(w, f);
    else if (weighted) load_each<E, float>(static_cast<const float*>(p.weight) + u * E, f);
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = weighted ? v[e] * inv * f[e] : v[e] * inv;
  };
  // the warps' trip counts are uniform: a warp whose last rows run out works on a row of nothing
  for (uint32_t r0 = blockIdx.x * (kNormRopeThreads / kLanes) + (threadIdx.x >> 5) * kRows; r0 < rows; r0 += step) {
    const uint32_t r = r0 + ((threadIdx.x & 31) / kLanes);
    const bool here = r < rows;
    const uint32_t t = here ? r / (uint32_t)p.heads : 0, h = here ? r - t * (uint32_t)p.heads : 0;
    const T* x = static_cast<const T*>(p.x) + (int64_t)t * p.x_token + (int64_t)h * p.x_head;
    T* out = static_cast<T*>(p.out) + (int64_t)t * p.out_token + (int64_t)h * p.out_head;
    uint4 raw[kUnits], partner[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int u = lane + kLanes * i;
      raw[i] = here && u < units ? reinterpret_cast<const uint4*>(x)[u] : make_uint4(0u, 0u, 0u, 0u);
      if constexpr (!kInterleaved) {                    // the partners, half the rotated dims away
        const int o = u * E - p.rope_offset;
        partner[i] = make_uint4(0u, 0u, 0u, 0u);
        if (here && o >= 0 && o < p.rope_dim) partner[i] = reinterpret_cast<const uint4*>(x)[o < half ? u + half / E : u - half / E];
      }
    }
    const int pos = p.rope_dim ? __ldg(p.positions + t) : 0;
    const bool inside = p.rope_dim == 0 || (pos >= 0 && pos < p.max_positions);
    float inv = 1.f;
    if (p.norm) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        float v[E];
        unpack<T>(raw[i], v);
#pragma unroll
        for (int e = 0; e < E; ++e) ss = fmaf(v[e], v[e], ss);
      }
#pragma unroll
      for (int o = kLanes / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      inv = rsqrtf(ss / (float)p.dim + p.eps);
    }
    __syncwarp();                                     // in place: every lane has read its units and partners
    if (here && !inside && lane == 0 && p.err) atomicOr(p.err, SMLA_DEVERR_LEN_RANGE);
    const float* cs = p.cos_sin + (size_t)(inside ? pos : 0) * p.rope_dim;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int u = lane + kLanes * i, o = u * E - p.rope_offset;
      if (!here || u >= units) continue;
      float v[E];
      scaled(raw[i], wraw[i], u, inv, v);
      if (o >= 0 && o < p.rope_dim) {
        if constexpr (kInterleaved) {
          float c[E / 2], s[E / 2];
          load_table<E / 2>(cs + o / 2, c);
          load_table<E / 2>(cs + half + o / 2, s);
#pragma unroll
          for (int e = 0; e < E; e += 2) {
            const float a = v[e], b = v[e + 1];
            v[e] = a * c[e / 2] - b * s[e / 2];
            v[e + 1] = a * s[e / 2] + b * c[e / 2];
          }
        } else {
          const bool first = o < half;
          const int pu = first ? u + half / E : u - half / E, j = first ? o : o - half;
          float q[E], c[E], s[E];
          scaled(partner[i], narrow ? __ldg(static_cast<const uint4*>(p.weight) + pu) : wraw[i], pu, inv, q);
          load_table<E>(cs + j, c);
          load_table<E>(cs + half + j, s);
#pragma unroll
          for (int e = 0; e < E; ++e) v[e] = first ? v[e] * c[e] - q[e] * s[e] : q[e] * s[e] + v[e] * c[e];
        }
      }
      if (!inside)
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = 0.f;
      store_vec<E, T>(out + u * E, v);
    }
  }
}

template <typename T>
bool launch_norm_rope_wide(const NormRopeParams& p, cudaStream_t stream) {
  constexpr int E = 16 / sizeof(T);
  auto whole = [&](const void* q, int64_t a, int64_t b) {
    return reinterpret_cast<uintptr_t>(q) % 16 == 0 && a % E == 0 && b % E == 0;
  };
  const int unit = p.interleaved ? E : 2 * E;           // a rotated half, or pairs, in whole units
  if (p.dim % E || p.rope_offset % E || p.rope_dim % unit || !whole(p.x, p.x_token, p.x_head) ||
      !whole(p.out, p.out_token, p.out_head) || (p.rope_dim && !whole(p.cos_sin, 0, 0)) ||
      (p.norm && p.weight && p.weight_dtype == p.dtype && !whole(p.weight, 0, 0)) ||
      (int64_t)p.tokens * p.heads > 0x7fffffff)
    return false;
  const int units = p.dim / E;
  auto go = [&](auto interleaved, auto plain, int lanes) {
    auto kernel = p.interleaved || p.rope_dim == 0 ? interleaved : plain;
    const int64_t per = kNormRopeThreads / lanes, want = ((int64_t)p.tokens * p.heads + per - 1) / per;
    const int64_t most = (int64_t)p.sms * 8;            // blocks of 256 threads resident at once, at most
    kernel<<<(int)(want < most ? want : most), kNormRopeThreads, 0, stream>>>(p);
    return true;
  };
#define SMLA_NORM_ROPE(lanes, n) go(norm_rope_kernel<T, lanes, n, true>, norm_rope_kernel<T, lanes, n, false>, lanes)
  // up to 32 units (256 elements of 16 bits) a row is eight lanes', so that short rows fill the warp
  if (units <= 8) return SMLA_NORM_ROPE(8, 1);
  if (units <= 16) return SMLA_NORM_ROPE(8, 2);
  if (units <= 24) return SMLA_NORM_ROPE(8, 3);
  if (units <= 32) return SMLA_NORM_ROPE(8, 4);
  if (units <= 64) return SMLA_NORM_ROPE(32, 2);
  if (units <= 96) return SMLA_NORM_ROPE(32, 3);
  if (units <= 128) return SMLA_NORM_ROPE(32, 4);
  if (units <= 160) return SMLA_NORM_ROPE(32, 5);
  return SMLA_NORM_ROPE(32, 8);
#undef SMLA_NORM_ROPE
}

}  // namespace

cudaError_t launch_kv_norm_append(const NormAppendParams& p, cudaStream_t stream) {
  if (p.tokens == 0) return cudaSuccess;
  const int esz = p.dtype == SMLA_FP32 ? 4 : 2;
  const bool wide = reinterpret_cast<uintptr_t>(p.latent) % 16 == 0 && (p.latent_stride * esz) % 16 == 0 &&
                    reinterpret_cast<uintptr_t>(p.rope) % (4 * esz) == 0 && p.rope_stride % 4 == 0 &&
                    reinterpret_cast<uintptr_t>(p.weight) % 16 == 0;
  const int want = (int)(((int64_t)p.tokens + 2 * kNormAppendWarps - 1) / (2 * kNormAppendWarps));
  const int blocks = want < p.sms * kNormAppendBlocksPerSm ? want : p.sms * kNormAppendBlocksPerSm;
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
  const bool wide = p.dtype == SMLA_BF16   ? launch_norm_rope_wide<__nv_bfloat16>(p, stream)
                    : p.dtype == SMLA_FP16 ? launch_norm_rope_wide<__half>(p, stream)
                                           : launch_norm_rope_wide<float>(p, stream);
  if (wide) return cudaGetLastError();
  const int64_t want = (rows + kNormRopeThreads / 32 - 1) / (kNormRopeThreads / 32);
  const int blocks = (int)(want < (1 << 20) ? want : (1 << 20));
  auto go = [&](auto kernel) { kernel<<<blocks, kNormRopeThreads, 0, stream>>>(p); };
  if (p.dtype == SMLA_BF16) go(norm_rope_any_kernel<__nv_bfloat16>);
  else if (p.dtype == SMLA_FP16) go(norm_rope_any_kernel<__half>);
  else go(norm_rope_any_kernel<float>);
  return cudaGetLastError();
}

}  // namespace smla
