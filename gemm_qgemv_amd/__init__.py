"""Dequantize-fused low-bit matrix-vector / matrix-matrix products, a fused
greedy (argmax) head and the embedding-row gather for AMD MI355X (gfx950),
with the serving-step operators between them: a paged key/value cache held in
4 bits (page plan, append, read-back, attention) and token log probabilities,
and microscaled (MX) 4- and 8-bit numbers with their products and the router,
sort and products of an experts' layer.

The computation lives in ``libqg.so`` (HIP kernels behind the C ABI of
``include/qg.h``); this package is its thin ctypes binding, plus the seeded
synthetic-input generator (``gemm_qgemv_amd.synth``) and device-buffer helpers
(``gemm_qgemv_amd.tensors``).
"""
from ._binding import (KVCache, QG_B1_G128, QG_BF16, QG_ERR_ALIAS, QG_ERR_ALIGN, QG_ERR_FORMAT,  # noqa: F401
                       QG_ERR_LAUNCH, QG_ERR_NULL, QG_ERR_SCRATCH, QG_ERR_SHAPE, QG_ERR_UNSUPPORTED,
                       QG_ERR_WORKSPACE, QG_F32, QG_I8_G64, QG_I8_ROW, QG_MAX_ARGMAX_BATCH, QG_MAX_GEMV_BATCH, QG_MAX_PLAN_BATCH,
                       QG_MAX_TOP, QG_OK, QG_OP_GEMM,
                       QG_OP_GEMV, QG_OP_GEMV_ARGMAX, QG_STATIC_SCRATCH_BYTES, QG_U4_G64, QG_WS_CONTROL_BYTES,
                       QGError, qg_abi_version, qg_status_str, qg_workspace_bytes, qembed, qgemm,
                       qgemv, qgemv_argmax, qgemv_argmax_noalloc, qkv_append, qkv_attn,
                       qkv_attn_workspace_bytes, qkv_cache_bytes, qkv_plan, qkv_read, qlogprobs,
                       qlogprobs_workspace_bytes, QMOE_MAX_EXPERTS, QMOE_MAX_TOP, QMX_E2M1, QMX_E4M3, QMX_MAX_K, QMX_MAX_M,
                       QMX_NONE, QMX_SILU_MUL, qmoe_combine, qmoe_gemm, qmoe_gemm_workspace_bytes, qmoe_plan,
                       qmoe_plan_workspace_bytes, qmoe_route, qmx_dequant, qmx_gemm, qmx_gemm_workspace_bytes,
                       qmx_quant, qmx_scale_pitch)
