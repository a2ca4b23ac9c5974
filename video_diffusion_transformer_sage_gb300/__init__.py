"""SageAttention2-style quantised non-causal attention for GB300 (sm_103a).

The compute path is the C-ABI CUDA library `_build/libsage_gb300.so` (include/sage.h; sage_paged.h,
sage_paged_tree.h and sage_paged_pool.h for the paged K/V cache); this package is its thin Python
binding (`_lib`) plus the seeded synthetic inputs (`synth`).  Build with `build.build()`.
"""
from ._lib import (PagedBatch, PagedKV, PagedPool, PagedTree, Quantized, SageError, dense_workspace, header_functions,
                   lib, make_view, pad128, paged_workspace, quant_scratch, sage_attn_dense_bf16,
                   sage_attn_dense_bf16_tc, sage_attn_fwd, sage_attn_fwd_quantized, sage_check_device_status,
                   sage_debug_qk_int32, sage_debug_wait_timeout, sage_measure_mma_rate, sage_paged_append,
                   sage_paged_attn, sage_paged_attn_tree, sage_paged_compact, sage_paged_copy, sage_paged_fork,
                   sage_paged_release, sage_paged_reserve, sage_paged_tree, sage_qk_rmsnorm_rope, sage_quant_qkv,
                   sage_quant_v, sage_smooth_quant_qk, sage_smooth_quant_qk_rmsnorm_rope, status_block, workspace)

__all__ = ["PagedBatch", "PagedKV", "PagedPool", "PagedTree", "Quantized", "SageError", "dense_workspace",
           "header_functions", "lib", "make_view", "pad128", "paged_workspace", "quant_scratch",
           "sage_attn_dense_bf16", "sage_attn_dense_bf16_tc", "sage_attn_fwd", "sage_attn_fwd_quantized",
           "sage_check_device_status", "sage_debug_qk_int32", "sage_debug_wait_timeout", "sage_measure_mma_rate",
           "sage_paged_append", "sage_paged_attn", "sage_paged_attn_tree", "sage_paged_compact", "sage_paged_copy",
           "sage_paged_fork", "sage_paged_release", "sage_paged_reserve", "sage_paged_tree", "sage_qk_rmsnorm_rope",
           "sage_quant_qkv", "sage_quant_v", "sage_smooth_quant_qk", "sage_smooth_quant_qk_rmsnorm_rope",
           "status_block", "workspace"]
