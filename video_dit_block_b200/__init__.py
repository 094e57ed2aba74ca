"""Training-free block-sparse self-attention for video DiTs, native to B200 (sm_100a),
with the norms, 8-bit projections and rotary positions of the block around it.

The compute path is a C-ABI CUDA library (include/sba.h, csrc/); this package is its
Python binding.  See `sba` for the calls.
"""
from .sba import (RopeTable, SbaError, attention, attention_compensated, attention_mean_compensated, attention_paired,
                  attention_to_shards, block_means, dense_attention, device_status, gather_tokens, int8_linear,
                  keep_count, keep_count_budget, keep_token_count, kmax_for, lib, lse_workspace_size,
                  mean_compensation_workspace_size, pair_query_blocks, pool_select, pool_select_lse,
                  pool_select_means, qk_norm_rope_pool, residual_norm, rope_frequencies, rotary, set_attention_kernel,
                  set_wait_limit, sparse_attention, token_prune, token_quantize, workspace_size)

__all__ = ["RopeTable", "SbaError", "attention", "attention_compensated", "attention_mean_compensated",
           "attention_paired", "attention_to_shards", "block_means", "dense_attention", "device_status", "gather_tokens",
           "int8_linear", "keep_count", "keep_count_budget", "keep_token_count", "kmax_for", "lib",
           "lse_workspace_size", "mean_compensation_workspace_size", "pair_query_blocks", "pool_select",
           "pool_select_lse", "pool_select_means", "qk_norm_rope_pool", "residual_norm", "rope_frequencies", "rotary",
           "set_attention_kernel", "set_wait_limit", "sparse_attention", "token_prune", "token_quantize",
           "workspace_size"]
