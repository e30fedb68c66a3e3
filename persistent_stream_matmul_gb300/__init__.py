"""GB300 (sm_103a) dense GEMM: C = A*B with fp16/bf16 inputs and fp32
accumulation, with data-parallel, persistent and Stream-K tile schedules.

The compute runs in ``libpsm_gemm.so`` (hand-written CUDA, C ABI in
include/gemm.h, include/gemm_moe.h and include/gemm_scaled.h).  This package is its ctypes binding plus the seeded operand
generator.  Loading the binding's functions fails loudly if the library is
not built: there is no CPU fallback.
"""
from ._binding import (  # noqa: F401
    GEMM_BF16, GEMM_COL_MAJOR, GEMM_E4M3, GEMM_E5M2, GEMM_F32, GEMM_NORM_MAX_HIDDEN, GEMM_QUANTIZE_BLOCKS,
    GEMM_QUANTIZE_COLS, GEMM_QUANTIZE_ROWS, GEMM_SCALED_OPT_CTAS, GEMM_SCALED_FEW, GEMM_SCALED_OPT_FORM,
    GEMM_SCALED_OPT_INJECT_GIVE_UP, GEMM_SCALED_STRAIGHT, GEMM_SCALED_TURNED, GEMM_SCALE_BLOCK, GEMM_SCALE_GROUP, GEMM_SCALE_VECTOR, GEMM_GROUPED_INNER, GEMM_GROUPED_OPT_CTAS,
    GEMM_GROUPED_OPT_INJECT_GIVE_UP, GEMM_GROUPED_ROWS, GEMM_INDEX_I32, GEMM_INDEX_I64,
    GEMM_MOE_MAX_EXPERTS, GEMM_SCHED_AUTO, GEMM_F16, GEMM_ROW_MAJOR, GEMM_SCHED_DATA_PARALLEL,
    GEMM_SCHED_PERSISTENT, GEMM_SCHED_SPLITK, GEMM_SCHED_STREAMK, GemmError, GroupedPlan, Plan, SCHEDULES,
    ScaledPlan,
    gemm_grouped_last_status, gemm_grouped_plan_create, gemm_grouped_plan_create_offline,
    gemm_grouped_plan_destroy, gemm_grouped_plan_get_info, gemm_grouped_plan_set_option,
    gemm_grouped_plan_units, gemm_grouped_run,
    gemm_grouped_workspace_size, gemm_last_status, gemm_moe_combine, gemm_moe_combine_grad,
    gemm_moe_dispatch, gemm_moe_dispatch_grad, gemm_moe_sort, gemm_moe_sort_workspace_size,
    gemm_plan_create, gemm_plan_create_offline, gemm_plan_destroy, gemm_plan_get_info,
    gemm_plan_set_option, gemm_plan_set_trace, gemm_plan_tile_coords, gemm_plan_units, gemm_run,
    gemm_rms_norm, gemm_rms_norm_grad, gemm_rms_norm_grad_workspace_size, gemm_scaled_last_status,
    gemm_scaled_plan_create, gemm_scaled_plan_create_offline, gemm_scaled_plan_destroy, gemm_scaled_plan_get_info,
    gemm_scaled_plan_set_option, gemm_scaled_quantize, gemm_scaled_quantize_both,
    gemm_scaled_run, gemm_scaled_workspace_size,
    gemm_run_host, gemm_run_no_alloc, gemm_status_string, gemm_workspace_size, load,
)
