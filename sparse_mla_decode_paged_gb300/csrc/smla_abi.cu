// C-ABI entry points: argument checks on the host, then kernel launches on
// the caller's stream.  No allocation, no synchronisation (except
// sparse_mla_read_errors).
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "smla_internal.h"

using namespace smla;

namespace {

std::atomic<uint64_t> g_wait_limit_ns{kDefaultWaitNs};

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace

namespace smla {

uint64_t split_wait_limit_ns() { return g_wait_limit_ns.load(std::memory_order_relaxed); }

int check_decode_dims(const smla_dims* d) {
  if (!d) return SMLA_ERR_INVALID_ARG;
  if (d->batch < 1 || d->topk < 1 || d->max_pages_per_seq < 1 || d->num_pages < 1 || d->nsplit < 0)
    return SMLA_ERR_INVALID_ARG;
  if (d->heads_per_cta != 0 && !split_heads_supported(d->heads_per_cta)) return SMLA_ERR_INVALID_ARG;
  if (d->queries_per_request < 0 || (d->queries_per_request > 1 && d->batch % d->queries_per_request != 0))
    return SMLA_ERR_INVALID_ARG;
  if (d->merge < 0 || d->merge > 2) return SMLA_ERR_INVALID_ARG;
  if (d->page_size != kPageSize || d->d_latent != kDLatent || d->d_rope != kDRope) return SMLA_ERR_UNSUPPORTED;
  if (d->topk > kMaxTopk || d->nsplit > kMaxSplit || d->batch > kMaxBatch) return SMLA_ERR_UNSUPPORTED;
  if (!split_shape_supported(d->num_heads, d->topk)) return SMLA_ERR_UNSUPPORTED;
  return SMLA_OK;
}

}  // namespace smla

namespace {

int check_dims(const smla_dims* d) { return check_decode_dims(d); }

int check_inputs(const void* q, const void* kv, const int32_t* bt, const int32_t* topk, const int32_t* seq) {
  if (!q || !kv || !bt || !topk || !seq) return SMLA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(kv, 16) || !aligned(bt, 4) || !aligned(topk, 4) || !aligned(seq, 4))
    return SMLA_ERR_INVALID_ARG;
  return SMLA_OK;
}

bool dtype_known(int32_t t) { return t == SMLA_BF16 || t == SMLA_FP16 || t == SMLA_FP32; }
uintptr_t dtype_size(int32_t t) { return t == SMLA_FP32 ? 4 : 2; }
bool weight_dtype_ok(int32_t w, int32_t x) { return w == x || w == SMLA_FP32; }
bool eps_ok(float eps) { return eps >= 0.f && eps < INFINITY; }     // false for a NaN

constexpr int kMaxDevices = 64;

// SM count of the current device (queried once per device, then read from a per-device slot).
int sm_count_of_current_device(int* sms) {
  static std::atomic<int> cached[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SMLA_ERR_CUDA;
  if (dev >= 0 && dev < kMaxDevices) {
    const int c = cached[dev].load(std::memory_order_relaxed);
    if (c > 0) {
      *sms = c;
      return SMLA_OK;
    }
  }
  if (cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return SMLA_ERR_CUDA;
  if (dev >= 0 && dev < kMaxDevices) cached[dev].store(*sms, std::memory_order_relaxed);
  return SMLA_OK;
}

bool same_dims(const smla_dims& a, const smla_dims& b) {
  return a.batch == b.batch && a.num_heads == b.num_heads && a.topk == b.topk && a.page_size == b.page_size &&
         a.max_pages_per_seq == b.max_pages_per_seq && a.d_latent == b.d_latent && a.d_rope == b.d_rope &&
         a.nsplit == b.nsplit && a.num_pages == b.num_pages && a.heads_per_cta == b.heads_per_cta &&
         a.queries_per_request == b.queries_per_request && a.merge == b.merge;
}

// The scheduler's plan for dims with nsplit fixed (> 0) or chosen (0), on the current device.  The
// plan of the last call on this host thread is kept: a call with the same dims on a device with the
// same SM count reuses it.
int plan_on_current_device(const smla_dims* dims, int nsplit, smla_plan* plan) {
  struct Last {
    bool valid;
    int sms;
    smla_dims d;
    smla_plan plan;
  };
  thread_local Last last{};
  int sms = 0;
  const int st = sm_count_of_current_device(&sms);
  if (st != SMLA_OK) return st;
  smla_dims d = *dims;
  d.nsplit = nsplit;
  if (last.valid && last.sms == sms && same_dims(last.d, d)) {
    *plan = last.plan;
    return SMLA_OK;
  }
  const int r = sparse_mla_plan_for(&d, sms, plan);
  if (r == SMLA_OK) last = Last{true, sms, d, *plan};
  return r;
}

SplitParams make_params(const smla_dims* d, int nsplit, int nh, const void* q, const void* kv, const int32_t* bt,
                        const int32_t* topk, const int32_t* seq, float sm_scale) {
  SplitParams p{};
  p.q = static_cast<const uint16_t*>(q);
  p.kv = static_cast<const uint8_t*>(kv);
  p.block_table = bt;
  p.topk = topk;
  p.seq_lens = seq;
  p.sm_scale = sm_scale;
  p.B = d->batch;
  p.H = d->num_heads;
  p.topk_n = d->topk;
  p.max_pages = d->max_pages_per_seq;
  p.num_pages = d->num_pages;
  p.nsplit = nsplit;
  p.nh = nh;
  p.q_per_req = d->queries_per_request > 1 ? d->queries_per_request : 1;
  p.split_len = (d->topk + nsplit - 1) / nsplit;
  p.wait_ns = split_wait_limit_ns();
  return p;
}

// The whole decode (split kernel, then the merge when nsplit > 1); rows_out (may be null) receives the
// row the split kernel's gather warps resolved for every top-k entry.
int decode_impl(const smla_dims* dims, const void* q, const void* kv_cache, const int32_t* block_table,
                const int32_t* topk_idx, const int32_t* seq_lens, float sm_scale, void* out, float* lse,
                void* workspace, size_t workspace_bytes, int64_t* rows_out, cudaStream_t s) {
  int st = check_dims(dims);
  if (st != SMLA_OK) return st;
  st = check_inputs(q, kv_cache, block_table, topk_idx, seq_lens);
  if (st != SMLA_OK) return st;
  if (!out || !lse || !aligned(out, 16) || !aligned(lse, 4)) return SMLA_ERR_INVALID_ARG;
  if (rows_out && !aligned(rows_out, 8)) return SMLA_ERR_INVALID_ARG;
  // a fixed split count fixes the workspace size: checked before the device is queried for the plan
  if (dims->nsplit > 0) {
    const size_t need = workspace_bytes_for(dims->batch, dims->num_heads, dims->nsplit);
    if (!workspace || workspace_bytes < need || !aligned(workspace, 256)) return SMLA_ERR_WORKSPACE;
  }
  smla_plan plan;
  st = plan_on_current_device(dims, dims->nsplit, &plan);
  if (st != SMLA_OK) return st;
  const int nsplit = plan.nsplit;
  const size_t need = workspace_bytes_for(dims->batch, dims->num_heads, nsplit);
  if (!workspace || workspace_bytes < need || !aligned(workspace, 256)) return SMLA_ERR_WORKSPACE;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  SplitParams p = make_params(dims, nsplit, plan.heads_per_cta, q, kv_cache, block_table, topk_idx, seq_lens,
                              sm_scale);
  p.err = reinterpret_cast<uint32_t*>(ws);
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.rows_out = rows_out;
  p.final_out = (nsplit == 1);
  p.fused = plan.fused != 0;
  if (nsplit > 1) {
    const size_t lse_bytes = ((size_t)dims->batch * nsplit * dims->num_heads * sizeof(float) + 255) / 256 * 256;
    p.lse_part = reinterpret_cast<float*>(ws + kWorkspaceHeader);
    p.o_part = reinterpret_cast<float*>(ws + kWorkspaceHeader + lse_bytes);
  }
  if (launch_split(p, s) != cudaSuccess) return SMLA_ERR_CUDA;
  if (nsplit > 1 && !p.fused &&
      launch_combine(dims->batch, dims->num_heads, nsplit, p.o_part, p.lse_part, p.out, lse, s) != cudaSuccess)
    return SMLA_ERR_CUDA;
  return SMLA_OK;
}

}  // namespace

extern "C" int sparse_mla_plan(const smla_dims* dims, int32_t device, smla_plan* plan) {
  if (!dims || !plan || device < 0) return SMLA_ERR_INVALID_ARG;
  int sms = 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) return SMLA_ERR_CUDA;
  return sparse_mla_plan_for(dims, sms, plan);
}

extern "C" int sparse_mla_split(const smla_dims* dims, int32_t nsplit, const void* q, const void* kv_cache,
                                const int32_t* block_table, const int32_t* topk_idx, const int32_t* seq_lens,
                                float sm_scale, float* o_part, float* lse_part, uint32_t* err_word,
                                smla_stream_t stream) {
  int st = check_dims(dims);
  if (st != SMLA_OK) return st;
  st = check_inputs(q, kv_cache, block_table, topk_idx, seq_lens);
  if (st != SMLA_OK) return st;
  if (nsplit < 1 || nsplit > kMaxCombineSplit) return SMLA_ERR_INVALID_ARG;
  if (nsplit > kMaxSplit) return SMLA_ERR_UNSUPPORTED;
  if (!o_part || !lse_part || !aligned(o_part, 16) || !aligned(lse_part, 4)) return SMLA_ERR_INVALID_ARG;
  if (err_word && !aligned(err_word, 4)) return SMLA_ERR_INVALID_ARG;
  smla_plan plan;
  st = plan_on_current_device(dims, nsplit, &plan);
  if (st != SMLA_OK) return st;
  SplitParams p = make_params(dims, nsplit, plan.heads_per_cta, q, kv_cache, block_table, topk_idx, seq_lens,
                              sm_scale);
  p.o_part = o_part;
  p.lse_part = lse_part;
  p.err = err_word;
  p.final_out = false;
  return launch_split(p, (cudaStream_t)stream) == cudaSuccess ? SMLA_OK : SMLA_ERR_CUDA;
}

extern "C" int sparse_mla_decode(const smla_dims* dims, const void* q, const void* kv_cache,
                                 const int32_t* block_table, const int32_t* topk_idx, const int32_t* seq_lens,
                                 float sm_scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
                                 smla_stream_t stream) {
  return decode_impl(dims, q, kv_cache, block_table, topk_idx, seq_lens, sm_scale, out, lse, workspace,
                     workspace_bytes, nullptr, (cudaStream_t)stream);
}

extern "C" int sparse_mla_decode_rows(const smla_dims* dims, const void* q, const void* kv_cache,
                                      const int32_t* block_table, const int32_t* topk_idx, const int32_t* seq_lens,
                                      float sm_scale, void* out, float* lse, void* workspace,
                                      size_t workspace_bytes, int64_t* rows_out, smla_stream_t stream) {
  if (!rows_out) return SMLA_ERR_INVALID_ARG;
  return decode_impl(dims, q, kv_cache, block_table, topk_idx, seq_lens, sm_scale, out, lse, workspace,
                     workspace_bytes, rows_out, (cudaStream_t)stream);
}

extern "C" int sparse_mla_debug_set_wait_limit(uint64_t ns) {
  g_wait_limit_ns.store(ns ? ns : kDefaultWaitNs, std::memory_order_relaxed);
  return SMLA_OK;
}

extern "C" int sparse_mla_kv_append(const smla_append_dims* d, const void* latent, const void* rope,
                                    const int32_t* block_table, const int32_t* requests, const int32_t* positions,
                                    void* kv_cache, uint32_t* err_word, smla_stream_t stream) {
  if (!d) return SMLA_ERR_INVALID_ARG;
  if (d->tokens < 0 || d->num_requests < 1 || d->max_pages_per_seq < 1 || d->num_pages < 1)
    return SMLA_ERR_INVALID_ARG;
  if (d->page_size != kPageSize || d->d_latent != kDLatent || d->d_rope != kDRope) return SMLA_ERR_UNSUPPORTED;
  if (d->tokens > 0) {
    if (!latent || !rope || !block_table || !positions || !kv_cache) return SMLA_ERR_INVALID_ARG;
    if (!aligned(latent, 16) || !aligned(rope, 16) || !aligned(kv_cache, 16) || !aligned(block_table, 4) ||
        !aligned(positions, 4) || (requests && !aligned(requests, 4)))
      return SMLA_ERR_INVALID_ARG;
  }
  if (err_word && !aligned(err_word, 4)) return SMLA_ERR_INVALID_ARG;
  AppendParams p{};
  p.latent = static_cast<const uint16_t*>(latent);
  p.rope = static_cast<const uint16_t*>(rope);
  p.block_table = block_table;
  p.requests = requests;
  p.positions = positions;
  p.kv = static_cast<uint8_t*>(kv_cache);
  p.tokens = d->tokens;
  p.num_requests = d->num_requests;
  p.max_pages = d->max_pages_per_seq;
  p.num_pages = d->num_pages;
  p.err = err_word;
  return launch_kv_append(p, (cudaStream_t)stream) == cudaSuccess ? SMLA_OK : SMLA_ERR_CUDA;
}

extern "C" int sparse_mla_kv_norm_append(const smla_norm_append_dims* d, const void* latent, const void* rope,
                                         const void* norm_weight, float eps, const float* cos_sin,
                                         const int32_t* block_table, const int32_t* requests,
                                         const int32_t* positions, void* kv_cache, uint32_t* err_word,
                                         smla_stream_t stream) {
  if (!d) return SMLA_ERR_INVALID_ARG;
  if (d->tokens < 0 || d->num_requests < 1 || d->max_pages_per_seq < 1 || d->num_pages < 1 || d->max_positions < 1)
    return SMLA_ERR_INVALID_ARG;
  if (!dtype_known(d->dtype) || !weight_dtype_ok(d->weight_dtype, d->dtype) || !eps_ok(eps) ||
      (d->interleaved != 0 && d->interleaved != 1))
    return SMLA_ERR_INVALID_ARG;
  if (d->page_size != kPageSize || d->d_latent != kDLatent || d->d_rope != kDRope) return SMLA_ERR_UNSUPPORTED;
  if (d->latent_stride < kDLatent || d->rope_stride < kDRope) return SMLA_ERR_INVALID_ARG;
  if (d->tokens > 0) {
    if (!latent || !rope || !norm_weight || !cos_sin || !block_table || !positions || !kv_cache)
      return SMLA_ERR_INVALID_ARG;
    const uintptr_t e = dtype_size(d->dtype);
    if (!aligned(latent, e) || !aligned(rope, e) || !aligned(norm_weight, dtype_size(d->weight_dtype)) ||
        !aligned(cos_sin, 16) || !aligned(kv_cache, 16) || !aligned(block_table, 4) || !aligned(positions, 4) ||
        (requests && !aligned(requests, 4)))
      return SMLA_ERR_INVALID_ARG;
  }
  if (err_word && !aligned(err_word, 4)) return SMLA_ERR_INVALID_ARG;
  NormAppendParams p{};
  p.latent = latent;
  p.rope = rope;
  p.weight = norm_weight;
  p.cos_sin = cos_sin;
  p.block_table = block_table;
  p.requests = requests;
  p.positions = positions;
  p.kv = static_cast<uint8_t*>(kv_cache);
  p.num_pages = d->num_pages;
  p.latent_stride = d->latent_stride;
  p.rope_stride = d->rope_stride;
  p.tokens = d->tokens;
  p.num_requests = d->num_requests;
  p.max_pages = d->max_pages_per_seq;
  p.max_positions = d->max_positions;
  p.dtype = d->dtype;
  p.weight_dtype = d->weight_dtype;
  p.interleaved = d->interleaved;
  p.eps = eps;
  p.err = err_word;
  if (d->tokens == 0) return SMLA_OK;
  const int st = sm_count_of_current_device(&p.sms);
  if (st != SMLA_OK) return st;
  return launch_kv_norm_append(p, (cudaStream_t)stream) == cudaSuccess ? SMLA_OK : SMLA_ERR_CUDA;
}

extern "C" int sparse_mla_norm_rope(const smla_norm_rope_dims* d, const void* x, const void* weight, float eps,
                                    const float* cos_sin, const int32_t* positions, void* out, uint32_t* err_word,
                                    smla_stream_t stream) {
  if (!d) return SMLA_ERR_INVALID_ARG;
  if (d->tokens < 0 || d->num_heads < 1 || d->head_dim < 1 || d->rope_dim < 0 || d->rope_dim % 2 != 0 ||
      d->rope_offset < 0 || (int64_t)d->rope_offset + d->rope_dim > d->head_dim)
    return SMLA_ERR_INVALID_ARG;
  if (!dtype_known(d->dtype) || !weight_dtype_ok(d->weight_dtype, d->dtype) || (d->norm != 0 && d->norm != 1) ||
      (d->interleaved != 0 && d->interleaved != 1) || !eps_ok(eps))
    return SMLA_ERR_INVALID_ARG;
  if (d->rope_dim > 0 && d->max_positions < 1) return SMLA_ERR_INVALID_ARG;
  if (d->head_dim > kMaxNormRopeDim) return SMLA_ERR_UNSUPPORTED;
  if (d->x_token_stride < 0 || d->x_head_stride < 0 || d->out_token_stride < 0 || d->out_head_stride < 0)
    return SMLA_ERR_INVALID_ARG;
  // rows of out must not overlap: the smaller stride covers a row, the larger one every row of the smaller
  if (d->tokens > 0) {
    const bool token_outer = d->out_token_stride >= d->out_head_stride;
    const int64_t inner = token_outer ? d->out_head_stride : d->out_token_stride;
    const int64_t outer = token_outer ? d->out_token_stride : d->out_head_stride;
    const int64_t n_inner = token_outer ? d->num_heads : d->tokens, n_outer = token_outer ? d->tokens : d->num_heads;
    if (n_inner > 1 && inner < d->head_dim) return SMLA_ERR_INVALID_ARG;
    const int64_t span = (n_inner > 1 ? (n_inner - 1) * inner : 0) + d->head_dim;
    if (n_outer > 1 && outer < (n_inner > 1 ? span : d->head_dim)) return SMLA_ERR_INVALID_ARG;
    if (!x || !out || (d->rope_dim > 0 && (!cos_sin || !positions))) return SMLA_ERR_INVALID_ARG;
    const uintptr_t e = dtype_size(d->dtype);
    if (!aligned(x, e) || !aligned(out, e) || (weight && !aligned(weight, dtype_size(d->weight_dtype))) ||
        (cos_sin && !aligned(cos_sin, 4)) || (positions && !aligned(positions, 4)))
      return SMLA_ERR_INVALID_ARG;
  }
  if (err_word && !aligned(err_word, 4)) return SMLA_ERR_INVALID_ARG;
  NormRopeParams p{};
  p.x = x;
  p.weight = weight;
  p.cos_sin = cos_sin;
  p.positions = positions;
  p.out = out;
  p.x_token = d->x_token_stride;
  p.x_head = d->x_head_stride;
  p.out_token = d->out_token_stride;
  p.out_head = d->out_head_stride;
  p.tokens = d->tokens;
  p.heads = d->num_heads;
  p.dim = d->head_dim;
  p.rope_dim = d->rope_dim;
  p.rope_offset = d->rope_offset;
  p.max_positions = d->max_positions;
  p.dtype = d->dtype;
  p.weight_dtype = d->weight_dtype;
  p.norm = d->norm;
  p.interleaved = d->interleaved;
  p.eps = eps;
  p.err = err_word;
  if (d->tokens == 0) return SMLA_OK;
  const int st = sm_count_of_current_device(&p.sms);
  if (st != SMLA_OK) return st;
  return launch_norm_rope(p, (cudaStream_t)stream) == cudaSuccess ? SMLA_OK : SMLA_ERR_CUDA;
}

extern "C" int sparse_mla_kv_read(const smla_append_dims* d, const void* kv_cache, const int32_t* block_table,
                                  const int32_t* requests, const int32_t* positions, void* out, int32_t out_dtype,
                                  uint32_t* err_word, smla_stream_t stream) {
  if (!d) return SMLA_ERR_INVALID_ARG;
  if (d->tokens < 0 || d->num_requests < 1 || d->max_pages_per_seq < 1 || d->num_pages < 1 || !dtype_known(out_dtype))
    return SMLA_ERR_INVALID_ARG;
  if (d->page_size != kPageSize || d->d_latent != kDLatent || d->d_rope != kDRope) return SMLA_ERR_UNSUPPORTED;
  if (d->tokens > 0) {
    if (!kv_cache || !block_table || !positions || !out) return SMLA_ERR_INVALID_ARG;
    if (!aligned(kv_cache, 16) || !aligned(out, 16) || !aligned(block_table, 4) || !aligned(positions, 4) ||
        (requests && !aligned(requests, 4)))
      return SMLA_ERR_INVALID_ARG;
  }
  if (err_word && !aligned(err_word, 4)) return SMLA_ERR_INVALID_ARG;
  ReadParams p{};
  p.kv = static_cast<const uint8_t*>(kv_cache);
  p.block_table = block_table;
  p.requests = requests;
  p.positions = positions;
  p.out = out;
  p.num_pages = d->num_pages;
  p.tokens = d->tokens;
  p.num_requests = d->num_requests;
  p.max_pages = d->max_pages_per_seq;
  p.out_dtype = out_dtype;
  p.err = err_word;
  return launch_kv_read(p, (cudaStream_t)stream) == cudaSuccess ? SMLA_OK : SMLA_ERR_CUDA;
}

extern "C" int sparse_mla_dense_plan(const smla_dense_dims* dims, int32_t device, smla_dense_plan* plan) {
  if (!dims || !plan || device < 0) return SMLA_ERR_INVALID_ARG;
  int sms = 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) return SMLA_ERR_CUDA;
  return sparse_mla_dense_plan_for(dims, sms, plan);
}

namespace {
// What a masked decode adds to a dense one.
struct ScoreForm {
  float softcap = 0.f;
  const float* slopes = nullptr;
  const int32_t* starts = nullptr;
  const int32_t* prefix_lens = nullptr;
};

int dense_decode(const smla_dense_dims* d, const ScoreForm& form, const void* q, const void* kv_cache,
                 const int32_t* block_table, const int32_t* seq_lens, float sm_scale, void* out, float* lse, void* workspace,
                 size_t workspace_bytes, smla_stream_t stream) {
  // the checks that need no device come first; the workspace's size and what a CTA can count depend on its SMs
  smla_dense_plan plan;
  int st = sparse_mla_dense_plan_for(d, kDenseMaxCtas, &plan);
  if (st != SMLA_OK) return st;
  st = check_inputs(q, kv_cache, block_table, seq_lens, seq_lens);
  if (st != SMLA_OK) return st;
  if (!out || !lse || !aligned(out, 16) || !aligned(lse, 4)) return SMLA_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < kWorkspaceHeader || !aligned(workspace, 256)) return SMLA_ERR_WORKSPACE;
  int sms = 0;
  st = sm_count_of_current_device(&sms);
  if (st != SMLA_OK) return st;
  st = sparse_mla_dense_plan_for(d, sms, &plan);
  if (st != SMLA_OK) return st;
  if (workspace_bytes < plan.workspace_bytes) return SMLA_ERR_WORKSPACE;
  DenseParams p{};
  p.q = static_cast<const uint16_t*>(q);
  p.kv = static_cast<const uint8_t*>(kv_cache);
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.sm_scale = sm_scale;
  p.B = d->batch;
  p.H = d->num_heads;
  p.q_per_req = d->queries_per_request > 1 ? d->queries_per_request : 1;
  p.max_pages = d->max_pages_per_seq;
  p.num_pages = d->num_pages;
  p.requests = p.B / p.q_per_req;
  p.nr = plan.rows_per_cta;
  p.groups = plan.row_groups;
  p.ctas = plan.ctas;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.err = static_cast<uint32_t*>(workspace);
  p.softcap = form.softcap;
  p.slopes = form.slopes;
  p.starts = form.starts;
  p.prefix_lens = form.prefix_lens;
  p.wait_ns = split_wait_limit_ns();
  return launch_dense(p, (cudaStream_t)stream) == cudaSuccess ? SMLA_OK : SMLA_ERR_CUDA;
}
}  // namespace

extern "C" int sparse_mla_dense_decode(const smla_dense_dims* d, const void* q, const void* kv_cache,
                                       const int32_t* block_table, const int32_t* seq_lens, float sm_scale, void* out,
                                       float* lse, void* workspace, size_t workspace_bytes, smla_stream_t stream) {
  return dense_decode(d, ScoreForm{}, q, kv_cache, block_table, seq_lens, sm_scale, out, lse, workspace, workspace_bytes,
                      stream);
}

extern "C" int sparse_mla_masked_decode(const smla_dense_dims* d, const void* q, const void* kv_cache,
                                        const int32_t* block_table, const int32_t* seq_lens, float sm_scale, float softcap,
                                        const float* slopes, const int32_t* starts, const int32_t* prefix_lens, void* out,
                                        float* lse, void* workspace, size_t workspace_bytes, smla_stream_t stream) {
  // (a cap outside this range would leave the exponent's factor 2 / cap without bits; false for a NaN)
  if (!(softcap == 0.f || (softcap >= 0x1p-20f && softcap <= 0x1p20f))) return SMLA_ERR_INVALID_ARG;
  if ((prefix_lens && !starts) || (slopes && !aligned(slopes, 4)) || (starts && !aligned(starts, 4)) ||
      (prefix_lens && !aligned(prefix_lens, 4)))
    return SMLA_ERR_INVALID_ARG;
  ScoreForm form;
  form.softcap = softcap;
  form.slopes = slopes;
  form.starts = starts;
  form.prefix_lens = prefix_lens;
  return dense_decode(d, form, q, kv_cache, block_table, seq_lens, sm_scale, out, lse, workspace, workspace_bytes, stream);
}

extern "C" int sparse_mla_topk_select(const smla_topk_dims* d, const float* scores, const int32_t* seq_lens,
                                      int32_t* topk_idx, uint32_t* err_word, smla_stream_t stream) {
  if (!d) return SMLA_ERR_INVALID_ARG;
  if (d->batch < 0 || d->num_cols < 1 || d->row_stride < d->num_cols || d->k < 1 || d->cluster_ctas < 0 ||
      d->cluster_ctas > kTopkMaxCluster)
    return SMLA_ERR_INVALID_ARG;
  if (d->k > kMaxTopk || d->num_cols > kTopkMaxCluster * kTopkMaxChunk) return SMLA_ERR_UNSUPPORTED;
  if (d->batch > 0) {
    if (!scores || !seq_lens || !topk_idx) return SMLA_ERR_INVALID_ARG;
    if (!aligned(scores, 4) || !aligned(seq_lens, 4) || !aligned(topk_idx, 4)) return SMLA_ERR_INVALID_ARG;
  }
  if (err_word && !aligned(err_word, 4)) return SMLA_ERR_INVALID_ARG;
  if (d->batch == 0) return SMLA_OK;
  int sms = 0;
  const int st = sm_count_of_current_device(&sms);
  if (st != SMLA_OK) return st;
  TopkParams p{};
  if (!topk_plan(d->batch, d->num_cols, sms, d->cluster_ctas, &p.csize, &p.chunk)) return SMLA_ERR_UNSUPPORTED;
  p.scores = scores;
  p.seq_lens = seq_lens;
  p.out = topk_idx;
  p.err = err_word;
  p.stride = d->row_stride;
  p.num_cols = d->num_cols;
  p.k = d->k;
  p.vec4 = aligned(scores, 16) && d->row_stride % 4 == 0;
  return launch_topk(p, d->batch, (cudaStream_t)stream) == cudaSuccess ? SMLA_OK : SMLA_ERR_CUDA;
}

extern "C" int sparse_mla_topk_plan_for(const smla_topk_dims* d, int32_t sm_count, int32_t* cluster_ctas,
                                        int32_t* chunk_positions) {
  if (!d || !cluster_ctas || !chunk_positions || sm_count < 1) return SMLA_ERR_INVALID_ARG;
  if (d->batch < 0 || d->num_cols < 1 || d->row_stride < d->num_cols || d->k < 1 || d->cluster_ctas < 0 ||
      d->cluster_ctas > kTopkMaxCluster)
    return SMLA_ERR_INVALID_ARG;
  if (d->k > kMaxTopk || d->num_cols > kTopkMaxCluster * kTopkMaxChunk) return SMLA_ERR_UNSUPPORTED;
  int c = 0, ch = 0;
  if (!topk_plan(d->batch > 0 ? d->batch : 1, d->num_cols, sm_count, d->cluster_ctas, &c, &ch))
    return SMLA_ERR_UNSUPPORTED;
  *cluster_ctas = c;
  *chunk_positions = ch;
  return SMLA_OK;
}

extern "C" int sparse_mla_combine(int32_t batch, int32_t num_heads, int32_t nsplit, const float* o_part,
                                  const float* lse_part, void* out, float* lse, smla_stream_t stream) {
  if (batch < 1 || num_heads < 1 || nsplit < 1 || nsplit > kMaxCombineSplit) return SMLA_ERR_INVALID_ARG;
  if (!o_part || !lse_part || !out || !lse) return SMLA_ERR_INVALID_ARG;
  if (!aligned(o_part, 16) || !aligned(out, 8) || !aligned(lse_part, 4) || !aligned(lse, 4))
    return SMLA_ERR_INVALID_ARG;
  return launch_combine(batch, num_heads, nsplit, o_part, lse_part, static_cast<uint16_t*>(out), lse,
                        (cudaStream_t)stream) == cudaSuccess
             ? SMLA_OK
             : SMLA_ERR_CUDA;
}

extern "C" int sparse_mla_gather_rows(const smla_dims* dims, const int32_t* block_table, const int32_t* topk_idx,
                                      const int32_t* seq_lens, int64_t* rows_out, smla_stream_t stream) {
  if (!dims) return SMLA_ERR_INVALID_ARG;
  if (dims->batch < 1 || dims->topk < 1 || dims->max_pages_per_seq < 1 || dims->num_pages < 1)
    return SMLA_ERR_INVALID_ARG;
  if (dims->page_size != kPageSize) return SMLA_ERR_UNSUPPORTED;
  if (!block_table || !topk_idx || !seq_lens || !rows_out || !aligned(rows_out, 8)) return SMLA_ERR_INVALID_ARG;
  return launch_gather_rows(block_table, topk_idx, seq_lens, dims->batch, dims->topk, dims->max_pages_per_seq,
                            dims->num_pages, dims->queries_per_request > 1 ? dims->queries_per_request : 1, rows_out,
                            (cudaStream_t)stream) == cudaSuccess
             ? SMLA_OK
             : SMLA_ERR_CUDA;
}

extern "C" int sparse_mla_clear_errors(void* workspace, smla_stream_t stream) {
  if (!workspace) return SMLA_ERR_INVALID_ARG;
  return cudaMemsetAsync(workspace, 0, sizeof(uint32_t), (cudaStream_t)stream) == cudaSuccess ? SMLA_OK
                                                                                            : SMLA_ERR_CUDA;
}

extern "C" int sparse_mla_read_errors(const void* workspace, uint32_t* flags, smla_stream_t stream) {
  if (!workspace || !flags) return SMLA_ERR_INVALID_ARG;
  if (cudaMemcpyAsync(flags, workspace, sizeof(uint32_t), cudaMemcpyDeviceToHost, (cudaStream_t)stream) !=
      cudaSuccess)
    return SMLA_ERR_CUDA;
  return cudaStreamSynchronize((cudaStream_t)stream) == cudaSuccess ? SMLA_OK : SMLA_ERR_CUDA;
}

extern "C" const char* sparse_mla_status_string(int status) {
  switch (status) {
    case SMLA_OK: return "ok";
    case SMLA_ERR_INVALID_ARG: return "invalid argument";
    case SMLA_ERR_UNSUPPORTED: return "unsupported shape";
    case SMLA_ERR_WORKSPACE: return "workspace missing or too small";
    case SMLA_ERR_CUDA: return "CUDA error";
    default: return "unknown status";
  }
}

extern "C" int sparse_mla_attention_weights(const smla_weights_dims* d, const void* q, const void* kv_cache,
                                            const int32_t* block_table, const int32_t* seq_lens, const float* lse,
                                            float sm_scale, float decay, float* weights, uint32_t* err_word,
                                            smla_stream_t stream) {
  if (!d) return SMLA_ERR_INVALID_ARG;
  const int sq = d->queries_per_request > 1 ? d->queries_per_request : 1;
  if (d->batch < 0 || d->num_heads < 1 || d->max_pages_per_seq < 1 || d->num_pages < 1 || d->queries_per_request < 0 ||
      d->batch % sq != 0 || d->num_cols < 0 || !(decay >= 0.f && decay <= 3.0e38f))
    return SMLA_ERR_INVALID_ARG;
  const int requests = d->batch / sq;
  if (requests > 1 && d->weights_stride < d->num_cols) return SMLA_ERR_INVALID_ARG;
  if (d->page_size != kPageSize || d->d_latent != kDLatent || d->d_rope != kDRope) return SMLA_ERR_UNSUPPORTED;
  // a CTA counts its tiles, and a request its positions, in 32 bits
  if (d->batch > kMaxBatch || d->num_heads > kDenseMaxHeads || d->num_pages > 0x7fffffff || d->num_cols > kMaxCols)
    return SMLA_ERR_UNSUPPORTED;
  if (d->batch > 0 && d->num_cols > 0) {
    const int st = check_inputs(q, kv_cache, block_table, seq_lens, seq_lens);
    if (st != SMLA_OK) return st;
    if (!lse || !weights || !aligned(lse, 4) || !aligned(weights, 4)) return SMLA_ERR_INVALID_ARG;
  }
  if (err_word && !aligned(err_word, 4)) return SMLA_ERR_INVALID_ARG;
  if (d->batch == 0) return SMLA_OK;
  if (d->num_cols == 0) {                                   // lengths are checked all the same, for the error word
    if (!err_word || !seq_lens) return SMLA_OK;
    if (!aligned(seq_lens, 4)) return SMLA_ERR_INVALID_ARG;
  }
  int sms = 0;
  const int st = sm_count_of_current_device(&sms);
  if (st != SMLA_OK) return st;
  if ((int64_t)requests * ((d->num_cols + kDenseTile - 1) / kDenseTile) / sms >= 0x7fffffff) return SMLA_ERR_UNSUPPORTED;
  WeightsParams p{};
  p.q = static_cast<const uint16_t*>(q);
  p.kv = static_cast<const uint8_t*>(kv_cache);
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.lse = lse;
  p.weights = weights;
  p.sm_scale = sm_scale;
  p.decay = decay;
  p.H = d->num_heads;
  p.q_per_req = sq;
  p.requests = requests;
  p.max_pages = d->max_pages_per_seq;
  p.cols = d->num_cols;
  p.num_pages = d->num_pages;
  p.weights_stride = d->weights_stride;
  p.err = err_word;
  p.wait_ns = split_wait_limit_ns();
  return launch_weights(p, sms, (cudaStream_t)stream) == cudaSuccess ? SMLA_OK : SMLA_ERR_CUDA;
}

namespace {
// Records of a request that can move at most (half of its slots), and the workspace's parts.
int evict_list_len(const smla_evict_dims* d) { return d->num_cols / 2 + 1; }
size_t evict_moved_bytes(const smla_evict_dims* d) { return ((size_t)d->num_requests * 4 + 255) / 256 * 256; }
}  // namespace

extern "C" size_t sparse_mla_kv_evict_workspace_size(const smla_evict_dims* d) {
  if (!d || d->num_requests < 0 || d->num_cols < 0) return 0;
  return evict_moved_bytes(d) + (size_t)d->num_requests * 2 * evict_list_len(d) * 4;
}

extern "C" int sparse_mla_kv_evict(const smla_evict_dims* d, float* weights, int32_t* positions,
                                   const int32_t* next_positions, const int32_t* seq_lens, const int32_t* keep,
                                   void* kv_cache, const int32_t* block_table, int32_t* new_lens, void* workspace,
                                   size_t workspace_bytes, uint32_t* err_word, smla_stream_t stream) {
  if (!d) return SMLA_ERR_INVALID_ARG;
  if (d->num_requests < 0 || d->num_cols < 1 || d->max_pages_per_seq < 1 || d->num_pages < 1 || d->sinks < 0 ||
      d->recent < 0 || (!keep && d->keep < 0))
    return SMLA_ERR_INVALID_ARG;
  if (d->num_requests > 1 && (d->weights_stride < d->num_cols || d->positions_stride < d->num_cols))
    return SMLA_ERR_INVALID_ARG;
  if (d->page_size != kPageSize || d->d_latent != kDLatent || d->d_rope != kDRope) return SMLA_ERR_UNSUPPORTED;
  if (d->num_requests > kMaxBatch || d->num_cols > kMaxCols || d->num_pages > 0x7fffffff) return SMLA_ERR_UNSUPPORTED;
  if (err_word && !aligned(err_word, 4)) return SMLA_ERR_INVALID_ARG;
  if (d->num_requests == 0) return SMLA_OK;
  if (!weights || !positions || !next_positions || !seq_lens || !kv_cache || !block_table || !new_lens ||
      !aligned(weights, 4) || !aligned(positions, 4) || !aligned(next_positions, 4) || !aligned(seq_lens, 4) ||
      !aligned(kv_cache, 16) || !aligned(block_table, 4) || !aligned(new_lens, 4) || (keep && !aligned(keep, 4)))
    return SMLA_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < sparse_mla_kv_evict_workspace_size(d))
    return SMLA_ERR_WORKSPACE;
  int sms = 0;
  const int st = sm_count_of_current_device(&sms);
  if (st != SMLA_OK) return st;
  EvictParams p{};
  p.weights = weights;
  p.positions = positions;
  p.next_positions = next_positions;
  p.seq_lens = seq_lens;
  p.keep = keep;
  p.kv = static_cast<uint8_t*>(kv_cache);
  p.block_table = block_table;
  p.new_lens = new_lens;
  p.num_pages = d->num_pages;
  p.weights_stride = d->weights_stride;
  p.positions_stride = d->positions_stride;
  p.requests = d->num_requests;
  p.cols = d->num_cols;
  p.max_pages = d->max_pages_per_seq;
  p.keep_all = d->keep;
  p.sinks = d->sinks;
  p.recent = d->recent;
  p.list_len = evict_list_len(d);
  p.moved = static_cast<int32_t*>(workspace);
  p.lists = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + evict_moved_bytes(d));
  p.err = err_word;
  return launch_evict(p, sms, (cudaStream_t)stream) == cudaSuccess ? SMLA_OK : SMLA_ERR_CUDA;
}

namespace {

// The prefix kernel takes prefixes of at least so many rows, with tables of at least so many pages, in all not more than 4 GiB
// of expanded records (a call's workspace).  Measured, the dense kernel / the prefix kernel, whole calls: 64 rows x 1000 /
// 4096 / 65536 positions 21.1 / 18.7, 21.2 / 23.5, 40.9 / 56.7 us; 128 rows 21.1 / 18.7, 23.8 / 23.8, 57.9 / 57.4; 256 rows
// 22.2 / 19.2, 29.6 / 24.9, 87 / 65; 1024 rows 34 / 28, 45 / 35, 260 / 145.  (Shorter ones keep the dense kernel's exact keys.)
constexpr int64_t kPairsLeastRows = 128, kPairsLeastPages = 16, kPairsMostTiles = ((int64_t)4 << 30) / (9 * 16384);
// The requests' own tables go along while all that is expanded stays within 5 GiB.
constexpr int64_t kPairsMostAll = ((int64_t)5 << 30) / (9 * 16384);

// How a shared decode runs on a device with `sms` SMs.
struct SharedPlan {
  int nr, own_groups, prefix_groups;
  bool pairs;                              // the prefix kernel takes the prefixes
  bool own;                                // and the requests' own positions
  int row_blocks, tiles_per_prefix, own_blocks, tiles_per_own;
  size_t results_at, lse_at, slots_at, slots_lse_at, info_at, begins_at, expanded_at, bytes;  // behind the dense decode's
};

int shared_plan(const smla_shared_dims* d, int sms, SharedPlan* plan) {
  if (!d || sms < 1) return SMLA_ERR_INVALID_ARG;
  const int sq = d->queries_per_request > 1 ? d->queries_per_request : 1;
  if (d->batch < 1 || d->num_heads < 1 || d->max_pages_per_seq < 1 || d->prefix_pages < 1 || d->num_prefixes < 1 ||
      d->num_pages < 1 || d->queries_per_request < 0 || d->batch % sq != 0 || d->batch / sq % d->num_prefixes != 0)
    return SMLA_ERR_INVALID_ARG;
  if (d->page_size != kPageSize || d->d_latent != kDLatent || d->d_rope != kDRope) return SMLA_ERR_UNSUPPORTED;
  if (d->batch > kMaxBatch || d->num_heads > kDenseMaxHeads || d->num_pages > 0x7fffffff) return SMLA_ERR_UNSUPPORTED;
  const int ctas = sms < kDenseMaxCtas ? sms : kDenseMaxCtas;
  const int64_t requests = d->batch / sq, rows = (int64_t)sq * d->num_heads, all = (int64_t)d->batch * d->num_heads;
  const int64_t prefix_rows = all / d->num_prefixes;
  plan->tiles_per_prefix = (int)((d->prefix_pages + (int64_t)1) / 2);
  plan->tiles_per_own = (int)((d->max_pages_per_seq + (int64_t)1) / 2);
  plan->pairs = prefix_rows >= kPairsLeastRows && d->prefix_pages >= kPairsLeastPages && sms >= 2 &&
                (int64_t)d->num_prefixes * plan->tiles_per_prefix <= kPairsMostTiles;
  auto tiles = [&](int nr) {
    return requests * ((rows + nr - 1) / nr) * ((d->max_pages_per_seq + (int64_t)1) / 2) +
           (plan->pairs ? 0 : d->num_prefixes * ((prefix_rows + nr - 1) / nr) * plan->tiles_per_prefix);
  };
  plan->nr = dense_rows_per_cta(plan->pairs ? rows : prefix_rows, ctas, tiles(16), tiles(32));
  if (tiles(plan->nr) / ctas >= 0x7fffffff) return SMLA_ERR_UNSUPPORTED;     // a CTA counts its tiles in 32 bits
  plan->own_groups = (int)((rows + plan->nr - 1) / plan->nr);
  plan->prefix_groups = (int)((prefix_rows + plan->nr - 1) / plan->nr);
  plan->results_at = dense_workspace_bytes(ctas, plan->nr);
  plan->lse_at = plan->results_at + (size_t)2 * all * kDLatent * sizeof(float);
  plan->bytes = plan->lse_at + (size_t)2 * all * sizeof(float);
  plan->own = false;
  if (plan->pairs) {
    auto after = [](size_t at) { return (at + 255) / 256 * 256; };
    const int64_t pairs = ctas / 2, all_tiles = (int64_t)d->num_prefixes * plan->tiles_per_prefix;
    plan->row_blocks = (int)((prefix_rows + 127) / 128);
    plan->own_blocks = (int)((rows + 127) / 128);
    const int64_t work = all_tiles * plan->row_blocks, own_tiles = requests * plan->tiles_per_own;
    if (work / pairs >= 0x7fffffff) return SMLA_ERR_UNSUPPORTED;
    plan->own = own_tiles * plan->own_blocks <= (work / 4 > 2 * pairs ? work / 4 : 2 * pairs) &&
                all_tiles + own_tiles <= kPairsMostAll;
    const size_t pages = 2 * (size_t)(all_tiles + (plan->own ? own_tiles : 0));
    plan->slots_at = after(plan->bytes);
    plan->slots_lse_at = plan->slots_at + 2 * pairs * 128 * kDLatent * sizeof(float);
    plan->begins_at = after(plan->slots_lse_at + 2 * pairs * 128 * sizeof(float));
    plan->info_at = after(plan->begins_at + (size_t)(d->num_prefixes + requests + 2) * sizeof(long long));
    plan->expanded_at = after(plan->info_at + 2 * pages * sizeof(int4));
    plan->bytes = plan->expanded_at + pages * 9 * 8192;
  }
  return SMLA_OK;
}

}  // namespace

extern "C" int sparse_mla_shared_workspace_size(const smla_shared_dims* d, int32_t sm_count, size_t* bytes) {
  SharedPlan plan;
  if (!bytes) return SMLA_ERR_INVALID_ARG;
  const int st = shared_plan(d, sm_count, &plan);
  if (st == SMLA_OK) *bytes = plan.bytes;
  return st;
}

extern "C" int sparse_mla_shared_decode(const smla_shared_dims* d, const void* q, const void* kv_cache,
                                        const int32_t* prefix_table, const int32_t* prefix_lens, const int32_t* block_table,
                                        const int32_t* seq_lens, float sm_scale, void* out, float* lse, void* workspace,
                                        size_t workspace_bytes, smla_stream_t stream) {
  SharedPlan plan;
  int st = shared_plan(d, kDenseMaxCtas, &plan);
  if (st != SMLA_OK) return st;
  st = check_inputs(q, kv_cache, block_table, seq_lens, seq_lens);
  if (st != SMLA_OK) return st;
  if (!prefix_table || !prefix_lens || !aligned(prefix_table, 4) || !aligned(prefix_lens, 4)) return SMLA_ERR_INVALID_ARG;
  if (!out || !lse || !aligned(out, 16) || !aligned(lse, 4)) return SMLA_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < kWorkspaceHeader || !aligned(workspace, 256)) return SMLA_ERR_WORKSPACE;
  int sms = 0;
  st = sm_count_of_current_device(&sms);
  if (st != SMLA_OK) return st;
  st = shared_plan(d, sms, &plan);
  if (st != SMLA_OK) return st;
  if (workspace_bytes < plan.bytes) return SMLA_ERR_WORKSPACE;
  SharedParams s{};
  DenseParams& p = s.dense;
  p.q = static_cast<const uint16_t*>(q);
  p.kv = static_cast<const uint8_t*>(kv_cache);
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.sm_scale = sm_scale;
  p.B = d->batch;
  p.H = d->num_heads;
  p.q_per_req = d->queries_per_request > 1 ? d->queries_per_request : 1;
  p.max_pages = d->max_pages_per_seq;
  p.num_pages = d->num_pages;
  p.requests = p.B / p.q_per_req;
  p.nr = plan.nr;
  p.groups = plan.own_groups;
  p.ctas = sms < kDenseMaxCtas ? sms : kDenseMaxCtas;
  p.shared_table = prefix_table;
  p.shared_lens = prefix_lens;
  p.prefixes = d->num_prefixes;
  p.shared_pages = d->prefix_pages;
  p.prefix_rows = p.B / d->num_prefixes * p.H;
  p.prefix_groups = plan.prefix_groups;
  p.out32 = reinterpret_cast<float*>(static_cast<char*>(workspace) + plan.results_at);
  p.lse32 = reinterpret_cast<float*>(static_cast<char*>(workspace) + plan.lse_at);
  p.err = static_cast<uint32_t*>(workspace);
  p.wait_ns = split_wait_limit_ns();
  PrefixParams& x = s.prefix;                                  // (what the join needs in any case first)
  x.prefixes = d->num_prefixes;
  x.rows = p.prefix_rows;
  x.requests = p.requests;
  x.q_per_req = p.q_per_req;
  x.H = p.H;
  x.all_rows = (size_t)p.B * p.H;
  x.out32 = p.out32;
  x.lse32 = p.lse32;
  if (plan.pairs) {
    char* ws = static_cast<char*>(workspace);
    x.q = p.q;
    x.kv = p.kv;
    x.table = prefix_table;
    x.lens = prefix_lens;
    x.num_pages = p.num_pages;
    x.sm_scale = sm_scale;
    x.pages = d->prefix_pages;
    x.row_blocks = plan.row_blocks;
    x.tiles_per_prefix = plan.tiles_per_prefix;
    x.own = plan.own;
    x.own_table = block_table;
    x.own_lens = seq_lens;
    x.own_pages = p.max_pages;
    x.own_blocks = plan.own_blocks;
    x.tiles_per_own = plan.tiles_per_own;
    x.pairs = p.ctas / 2;
    x.expanded = reinterpret_cast<unsigned char*>(ws + plan.expanded_at);
    x.info = reinterpret_cast<int4*>(ws + plan.info_at);
    x.begins = reinterpret_cast<long long*>(ws + plan.begins_at);
    x.slots = reinterpret_cast<float*>(ws + plan.slots_at);
    x.slots_lse = reinterpret_cast<float*>(ws + plan.slots_lse_at);
    x.err = p.err;
    x.wait_ns = p.wait_ns;
    p.prefixes = p.prefix_groups = p.shared_pages = 0;       // the dense kernel has the requests' own positions at most
  }
  s.out = static_cast<uint16_t*>(out);
  s.lse = lse;
  return launch_shared(s, (cudaStream_t)stream) == cudaSuccess ? SMLA_OK : SMLA_ERR_CUDA;
}
