"""fp8blk: fine-grained FP8 (1x128 activation tiles, 128x128 weight blocks)
quantization and block-scaled FP8 GEMM for MI355X (gfx950).

The compute lives in the HIP library built from ``csrc/`` (see ``build.py``);
``binding`` is its Python face.  ``inputs`` is the seeded synthetic input
generator.  Importing this package loads nothing; the library is loaded on
first use and its absence is an error.
"""
from .binding import (  # noqa: F401
    FP8_OUT_BF16, FP8_OUT_F32, Fp8Error, fp8_block_gemm, fp8_block_gemm_pow2,
    fp8_block_grouped_gemm, fp8_block_grouped_gemm_pow2, fp8_gemm_workspace_bytes,
    fp8_quant_act_1x128, fp8_quant_act_1x128_pow2, fp8_quant_weight_128x128,
    fp8_quant_weight_128x128_pow2, lib, status_string, fp8_quant_act_128x1_t,
    fp8_transpose_weight_128x128, fp8_block_gemm_wgrad, fp8_block_gemm_fused_quant,
    fp8_block_gemm_noalloc, fp8_block_gemm_dgrad, fp8_fused_quant_workspace_bytes,
    fp8_fused_quant_kernel_workspace_bytes, fp8_quant_act_128x1_t_pow2,
    fp8_block_gemm_wgrad_pow2, fp8_block_gemm_dgrad_pow2,
)

_MOE = (
    "FP8_W4_F32_1X128", "FP8_W4_E8M0_1X32", "fp8_moe_sort", "fp8_moe_sort_workspace_bytes",
    "fp8_moe_dispatch", "fp8_moe_dispatch_quant_1x128", "fp8_moe_dispatch_quant_1x128_pow2",
    "fp8_moe_sort_dispatch", "fp8_moe_sort_dispatch_quant_1x128",
    "fp8_moe_sort_dispatch_quant_1x128_pow2", "fp8_moe_dispatch_grad", "fp8_moe_combine",
    "fp8_moe_combine_grad", "fp8_norm_residual", "fp8_norm_residual_quant_1x128",
    "fp8_norm_residual_quant_1x128_pow2", "fp8_norm_residual_grad",
    "fp8_norm_residual_grad_workspace_bytes", "fp8_w4_quant_1x128", "fp8_w4_quant_1x32",
    "fp8_w4_matvec", "fp8_w4_grouped_matvec",
)

_FFN = (
    "FP8_ACT_SILU", "FP8_ACT_GELU_TANH", "fp8_block_gemm_gated", "fp8_block_gemm_gated_pow2",
    "fp8_block_gemm_gated_quant_1x128", "fp8_block_gemm_gated_quant_1x128_pow2",
    "fp8_gated_gemm_workspace_bytes", "fp8_grouped_gated_gemm_workspace_bytes",
    "fp8_block_grouped_gemm_gated",
    "fp8_block_grouped_gemm_gated_pow2", "fp8_block_grouped_gemm_gated_quant_1x128",
    "fp8_block_grouped_gemm_gated_quant_1x128_pow2", "fp8_gated_grad",
    "fp8_gated_grad_quant_1x128", "fp8_gated_grad_quant_1x128_pow2", "fp8_gated_grad_quant",
    "fp8_gated_grad_quant_pow2", "fp8_dequant_act_1x128", "fp8_requant_act_128x1_t",
    "fp8_requant_act_128x1_t_pow2", "fp8_block_grouped_gemm_dgrad",
    "fp8_block_grouped_gemm_dgrad_pow2",
)


def __getattr__(name):
    """The operators around the expert products, from ``moe``, and inside a
    gated feed-forward block, from ``ffn``, on first use (they need torch, which
    importing this package does not load)."""
    if name in _MOE or name in _FFN:
        from . import ffn, moe
        value = getattr(moe if name in _MOE else ffn, name)
        globals()[name] = value
        return value
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")


def __dir__():
    return sorted(set(globals()) | set(_MOE) | set(_FFN))
