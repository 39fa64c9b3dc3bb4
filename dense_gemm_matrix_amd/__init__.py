"""Dense GEMM C = A*B for AMD MI355X (gfx950): hand-written HIP kernels behind a
C ABI (include/dgemm.h), with a thin ctypes binding of the same names; and the
linear layer's operators around it (_linear) and a feed-forward block's (_feedforward)."""
from ._binding import (  # noqa: F401
    DGEMM_ACT_NONE, DGEMM_ACT_RELU, DGEMM_ERR_ALIAS, DGEMM_ERR_DEVICE, DGEMM_ERR_INVALID_VALUE, DGEMM_ERR_LAUNCH,
    DGEMM_ERR_LEADING_DIM, DGEMM_ERR_MISALIGNED, DGEMM_ERR_SCRATCH_SIZE, DGEMM_ERR_TOO_LARGE, DGEMM_ERR_WORKSPACE,
    DGEMM_OK, DGEMM_STATIC_SCRATCH_BYTES,
    DGEMM_OUT_F32, DGEMM_OUT_SAME, DGEMM_PLAN_AUTO, DGEMM_PLAN_GRID, DGEMM_PLAN_STREAM_K,
    DGEMM_PLAN_NO_STREAM_K, LIB_PATH,
    DgemmError, dgemm_set_plan_override, dgemm_set_stream_k_wait_us, dgemm_status_string,
    dgemm_stream_k_schedule,
    dgemm_tile_map, gemm_bf16, gemm_ex, gemm_ex_plan, gemm_ex_static, gemm_f16, gemm_f32, gemm_f32_3xbf16,
    matmul, raw,
)
from ._linear import (  # noqa: F401
    ACT_CODES, gemm_act, gemm_act_bwd, gemm_act_bwd_workspace, gemm_act_plan, gemm_f8, gemm_f8_plan,
    linear, linear_backward, matmul_f8, quant_f8, quantize_f8, rms_norm, rms_norm_backward, rmsnorm,
    rmsnorm_bwd, rmsnorm_bwd_workspace,
)
from ._feedforward import (  # noqa: F401
    gemm_f8_block, gemm_f8_block_plan, gemm_gated, gemm_gated_bwd, gemm_gated_bwd_workspace, gemm_gated_plan,
    layer_norm, layer_norm_backward, layernorm, layernorm_bwd, layernorm_bwd_workspace, linear_gated,
    linear_gated_backward, matmul_f8_block, quant_f8_block, quantize_f8_block,
)
