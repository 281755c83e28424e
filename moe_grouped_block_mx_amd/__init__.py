"""Grouped block-scaled (MX) GEMM for MoE expert layers on AMD MI355X (gfx950).

The compute path is libmxgg.so (hand-written HIP kernels behind the C ABI of
include/mxgg.h); this package is its thin ctypes binding.
"""
from ._lib import (  # noqa: F401
    FORMATS, FP8_1x128, FP8_128x128, FP8_1x128_P2, FP8_128x128_P2, LAYOUT_BLOCK_MAJOR, LAYOUT_MASK, LAYOUT_MFMA,
    LAYOUT_ROW_MAJOR, KBLOCK_COLS, KBLOCK_MASK, KBLOCK_ROWS,
    I32, I64, INT8, LIB_PATH, MAX_EXPERTS, MXFP4, MXFP8, POW2_SCALES,
    MxggError, header_functions, lib,
    mxgg_grouped_dgrad, mxgg_grouped_fwd, mxgg_grouped_wgrad, mxgg_quantize_colwise_segpad, mxgg_quantize_dual,
    mxgg_mx_scale_stride, mxgg_mx_scales_relayout, mxgg_quantize_rowwise, mxgg_segpad_rows, mxgg_transpose_128x128,
    mxgg_workspace_size,
    BF16, F32, MOE_MAX_TOKENS, MOE_MAX_TOP_K, MOE_RENORMALIZE, MOE_W13_KBLOCK, MOE_W2_KBLOCK, NORM_L2, NORM_MAX,
    mxgg_clip_grad_norm, mxgg_clip_grads_with_norm, mxgg_grad_norm, mxgg_layer_norm_bwd, mxgg_layer_norm_fwd,
    mxgg_moe_layer,
    mxgg_dropout, mxgg_moe_combine, mxgg_moe_combine_bwd, mxgg_moe_dispatch, mxgg_moe_sort,
    dropout, moe_combine, moe_combine_bwd, moe_dispatch, moe_sort,
    clip_grad_norm, clip_grads_with_norm, grad_norm, layer_norm_bwd, layer_norm_fwd, moe_layer,
    grouped_dgrad, grouped_fwd, grouped_wgrad, quantize_colwise_segpad, quantize_dual, quantize_rowwise,
    mx_scale_stride, mx_scales_relayout, segpad_rows, transpose_128x128, workspace_size,
)
