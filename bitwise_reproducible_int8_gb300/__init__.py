"""Bitwise-reproducible int8 QAT linear layer (forward, backward) and its
fixed-order gradient reduction, for one GB300 (sm_103a).

The product is the C-ABI library ``librepro.so`` (declared in
``include/repro.h``); ``repro`` is its thin Python binding with the same
names.  ``inputs`` draws the seeded synthetic workloads.
"""
from .repro import (  # noqa: F401
    REPRO_BWD_DW_ACCUMULATE, REPRO_OK, REPRO_QMAX, REPRO_SCALE_ACT_AMAX,
    REPRO_SCALE_WEIGHT_MEANABS, ReproError, lib, repro_device_check, repro_grad_accum,
    repro_launch_count, repro_linear_bwd, repro_linear_bwd_ws_bytes, repro_linear_fwd,
    repro_linear_fwd_ws_bytes, repro_running_sum, repro_sumsq, repro_sumsq_ws_bytes,
    repro_adamw_step, repro_attn_bwd, repro_attn_bwd_ws_bytes, repro_attn_fwd, repro_attn_fwd_ws_bytes,
    repro_quant_i8, repro_quant_i8_multi, repro_wscale_multi, repro_wscale_multi_ws_bytes,
    repro_selftest, repro_set_launch_cfg, repro_state_hash, repro_state_hash_ws_bytes, repro_status_str,
    repro_treefold, repro_version, repro_wait_probe, repro_wscale, repro_wscale_ws_bytes,
    REPRO_HASH_LEAF_BYTES, REPRO_DEBUG_CHECK_FINITE, REPRO_ERR_NONFINITE, REPRO_ERR_TIMEOUT,
    repro_set_debug,
    REPRO_BF16, REPRO_DISTILL_BLOCK, REPRO_DISTILL_LOGPROBS, REPRO_DISTILL_STATS,
    REPRO_DISTILL_STAT_LSE, REPRO_EMBED_MAX_N, REPRO_EMBED_MAX_V, REPRO_ERR_INDEX, REPRO_F32, REPRO_I8,
    REPRO_QK_INTERLEAVED, REPRO_QK_MAX_D, repro_distill_bwd, repro_distill_fwd,
    repro_distill_ws_bytes, repro_embed_bwd, repro_embed_bwd_ws_bytes, repro_embed_fwd,
    repro_qk_norm_rope_bwd, repro_qk_norm_rope_bwd_ws_bytes, repro_qk_norm_rope_fwd,
    REPRO_MM_A_T, REPRO_MM_B_T, REPRO_MM_MAX_ROWS, REPRO_NORM_CHUNK, REPRO_NORM_GATE_ROWS,
    REPRO_NORM_MAX_D, REPRO_NORM_POST, REPRO_QUANT_COLUMNS, REPRO_SWIGLU_GROUP,
    repro_block_norm_bwd, repro_block_norm_bwd_ws_bytes, repro_block_norm_fwd, repro_matmul_i8,
    repro_matmul_i8_ws_bytes, repro_quant_rows_i8, repro_quant_rows_i8_ws_bytes, repro_swiglu_bwd,
    repro_swiglu_fwd,
)
