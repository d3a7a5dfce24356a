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
constexpr int kNormAppendBlocksPerSm = 16;

// One token of a warp, as loaded: latent dims 8 l .. 8 l + 7 and 256 + 8 l .. (blocks l / 16 and 2 + l / 16, so a
// block's amax is a reduction over 16 lanes, and every access of the warp is contiguous), rope dims 2 l, 2 l + 1, and
// the block-table entry.
struct AppendToken {
  float x[16], r0, r1;
  int pos, page;
};

template <typename T, bool kWide>
__device__ __forceinline__ AppendToken append_load(const NormAppendParams& p, int tok, int lane) {
  AppendToken a;
  const T* row = static_cast<const T*>(p.latent) + (int64_t)tok * p.latent_stride + 8 * lane;
  float (&lo)[8] = reinterpret_cast<float (&)[8]>(a.x[0]);
  float (&hi)[8] = reinterpret_cast<float (&)[8]>(a.x[8]);
  if constexpr (kWide) {
    load_vec<8, T>(row, lo);
    load_vec<8, T>(row + 256, hi);
  } else {
    load_each<8, T>(row, lo);
    load_each<8, T>(row + 256, hi);
  }
  const T* rr = static_cast<const T*>(p.rope) + (int64_t)tok * p.rope_stride + 2 * lane;
  a.r0 = to_f32<T>(rr[0]);
  a.r1 = to_f32<T>(rr[1]);
  const int req = p.requests ? __ldg(p.requests + tok) : tok;
  a.pos = __ldg(p.positions + tok);
  a.page = -1;
  if (req >= 0 && req < p.num_requests && a.pos >= 0 && (a.pos >> 6) < p.max_pages && a.pos < p.max_positions)
    a.page = __ldg(p.block_table + (size_t)req * p.max_pages + (a.pos >> 6));
  return a;
}

// One warp per token, the weights in registers over the warp's tokens.  What bounds it: HBM bytes (1152 read, 256 of
// cos and sin mostly from L2, 656 written per token of a 16-bit type).  Codes are n times the scale's reciprocal (one
// reciprocal per block; sixteen divisions per lane took half the kernel's issue slots).
template <typename T, bool kWide>
__global__ void __launch_bounds__(32 * kNormAppendWarps) kv_norm_append_kernel(const NormAppendParams p) {
  const int lane = threadIdx.x & 31;
  const int warps = gridDim.x * kNormAppendWarps;
  float w[16];
  load_weight<8, T>(p.weight, 8 * lane, p.weight_dtype, reinterpret_cast<float (&)[8]>(w[0]));
  load_weight<8, T>(p.weight, 256 + 8 * lane, p.weight_dtype, reinterpret_cast<float (&)[8]>(w[8]));
  for (int64_t tok = blockIdx.x * kNormAppendWarps + (threadIdx.x >> 5); tok < p.tokens; tok += warps) {
    AppendToken a = append_load<T, kWide>(p, (int)tok, lane);
    if (a.page < 0 || (int64_t)a.page >= p.num_pages) {
      if (lane == 0 && p.err) atomicOr(p.err, SMLA_DEVERR_PAGE_RANGE);
      continue;                                      // warp-uniform
    }
    unsigned char* rec = p.kv + ((int64_t)a.page * kPageSize + (a.pos & (kPageSize - 1))) * kRecordBytes;
    const float* cs = p.cos_sin + (size_t)a.pos * kDRope;

    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) ss = fmaf(a.x[i], a.x[i], ss);
#pragma unroll
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float inv = rsqrtf(ss * (1.f / kDLatent) + p.eps);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float* x = a.x + 8 * h;
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] = x[i] * inv * w[8 * h + i];
        amax = fmaxf(amax, fabsf(x[i]));
      }
#pragma unroll
      for (int o = 8; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      float scale = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
      if (scale == 0.f) scale = 1.f;                 // amax below the smallest float's 224 fold: codes of 0
      const bool tiny = scale < 0x1p-100f;           // its reciprocal may not be a float: both sides times 2^64
      const float up = __frcp_rn(tiny ? scale * 0x1p64f : scale);
      if (__builtin_expect(tiny, 0)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= 0x1p64f;
      }
      uint32_t c[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        c[i] = (uint32_t)f32x2_to_e4m3x2(x[4 * i] * up, x[4 * i + 1] * up) |
               ((uint32_t)f32x2_to_e4m3x2(x[4 * i + 2] * up, x[4 * i + 3] * up) << 16);
      reinterpret_cast<uint2*>(rec)[32 * h + lane] = make_uint2(c[0], c[1]);
      if ((lane & 15) == 0) reinterpret_cast<float*>(rec + kDLatent)[2 * h + (lane >> 4)] = scale;
    }

    float y0, y1;
    if (p.interleaved) {                             // this lane's two dims are pair `lane`
      const float co = __ldg(cs + lane), si = __ldg(cs + 32 + lane);
      y0 = a.r0 * co - a.r1 * si;
      y1 = a.r0 * si + a.r1 * co;
    } else {                                         // partners of dims 2 l, 2 l + 1 sit 16 lanes away
      const float q0 = __shfl_xor_sync(0xffffffffu, a.r0, 16), q1 = __shfl_xor_sync(0xffffffffu, a.r1, 16);
      const int j = (2 * lane) & 31;
      const float2 co = __ldg(reinterpret_cast<const float2*>(cs + j));
      const float2 si = __ldg(reinterpret_cast<const float2*>(cs + 32 + j));
      y0 = lane < 16 ? a.r0 * co.x - q0 * si.x : q0 * si.x + a.r0 * co.x;
      y1 = lane < 16 ? a.r1 * co.y - q1 * si.y : q1 * si.y + a.r1 * co.y;
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
  const bool wide = reinterpret_cast<uintptr_t>(p.latent) % 16 == 0 && (p.latent_stride * esz) % 16 == 0;
  const int want = (int)(((int64_t)p.tokens + kNormAppendWarps - 1) / kNormAppendWarps);
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
