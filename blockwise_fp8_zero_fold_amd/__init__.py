"""Python binding of libfp8z1 (the blockwise-FP8 ZeRO-1 shard step for MI355X).

Argument marshalling only: every step of the path runs in the HIP library.
The functions keep the C names of ``include/fp8z1.h``; tensors are passed
as device pointers, streams as ``torch.cuda.current_stream().cuda_stream``.
Importing this package loads the library and raises if it is not built.
"""
from ._lib import (  # noqa: F401
    ACT_GELU, ACT_NONE, ACT_SILU, ALL_RANKS, BF16, E4M3, F16, F32, GATE_CHANNEL, GATE_FULL, GATE_NONE, GATE_TOKEN,
    NOALLOC_MAX_SLOTS, ROUTE_MAX_CHOICES, ROUTE_MAX_EXPERTS, SCALE_AMAX, SCALE_POW2, SCORE_SIGMOID, SCORE_SOFTMAX,
    SPLIT_BLOCK, SPLIT_PARAM, STAT_PARTS,
    BLOCK_ENTRY_DTYPE, Ffn, Fp8z1Error, Hparams, Norm, Product, Routed, Router, State, Table,
    fp8z1_build_table, fp8z1_dequantize, fp8z1_encode_e4m3, fp8z1_ffn_down, fp8z1_ffn_down_bwd, fp8z1_ffn_up,
    fp8z1_ffn_bwd_weights, fp8z1_ffn_bwd_weights_workspace_bytes, fp8z1_ffn_up_bwd, fp8z1_ffn_wgrad, fp8z1_ffn_wgrad_workspace_bytes, fp8z1_ffn_workspace_bytes, fp8z1_fold, fp8z1_norm_join, fp8z1_norm_join8, fp8z1_norm_join_bwd,
    fp8z1_norm_join_bwd_workspace_bytes, fp8z1_state_init, fp8z1_state_read, fp8z1_state_write,
    fp8z1_ffn_up8, fp8z1_ffn_up8_workspace_bytes, fp8z1_linear, fp8z1_linear_bwd, fp8z1_linear_bwd_workspace_bytes,
    fp8z1_linear_workspace_bytes, fp8z1_combine, fp8z1_combine_bwd, fp8z1_dispatch, fp8z1_route, fp8z1_route_bwd, fp8z1_sort_tokens,
    fp8z1_sort_tokens_workspace_bytes, fp8z1_shard_sumsq, fp8z1_step, fp8z1_step_rowmajor, fp8z1_step_rowmajor_noalloc, fp8z1_step_workspace_bytes,
    fp8z1_unfold, fp8z1_probe_copy,
    fp8z1_probe_update_pattern, lib, lib_path,
)
