"""GB300 (sm_103a) sparse-MLA decode over a paged FP8 latent KV cache.

The compute runs in libsparse_mla.so (CUDA, C ABI in include/sparse_mla.h);
this package is its thin PyTorch binding plus the seeded workload generator.
"""
from .api import (alloc_dense_workspace, alloc_evict_workspace, alloc_shared_workspace, alloc_workspace,  # noqa: F401
                  clear_errors, dense_dims_of, dense_plan, dense_plan_for, dims_of, make_dense_dims, make_dims, plan,
                  plan_for, read_errors, rope_table, shared_dims_of, sparse_mla_attention_weights, sparse_mla_combine,
                  sparse_mla_decode, sparse_mla_dense_decode, sparse_mla_gather_rows, sparse_mla_kv_evict,
                  sparse_mla_kv_norm_append, sparse_mla_kv_read, sparse_mla_masked_decode, sparse_mla_norm_rope,
                  sparse_mla_shared_decode, sparse_mla_split, sparse_mla_topk_select, workspace_size)
