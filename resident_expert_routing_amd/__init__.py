"""MI355X-native routed-expert MoE layer against a partially resident expert arena.

The layer (TideLM README, "How adaptive expert loading works", items 1-3) runs
in libmoe_arena.so's HIP kernels for gfx950, behind the C ABI declared in
include/moe_arena.h.  `binding` wraps that ABI with ctypes; `runtime` adds the
torch plumbing (device buffers, arena upload).  Importing the package loads the
library and fails loudly if it has not been built.  `rows` has the batch's rows
in the order of the slots and back as differentiable functions, `int8` rows,
products and experts in 8-bit integers, `grouped` the experts' products in floating point
with gradients, `int4` products and experts with 4-bit weights.
"""
from . import binding
from .binding import (MOE_DT_BF16, MOE_DT_FP16, MOE_DT_FP32, MOE_OP_DEMAND, MOE_OP_EXPERTS, MOE_OP_HOT_PICK, MOE_OP_ROUTE, MoeError,
                      arena_load_slot, check, moe_combine, moe_combine_backward,
                      moe_demand_accumulate, moe_dispatch, moe_dispatch_backward,
                      moe_experts_forward, moe_grouped_matmul, moe_grouped_outer, moe_grouped_outer_ws_bytes,
                      moe_hot_install, moe_hot_pick, moe_int4_code_bytes, moe_int4_matmul,
                      moe_int4_quantize, moe_int4_scale_count, moe_mxfp4_row_bytes, moe_int8_matmul,
                      moe_int8_quantize, moe_int8_row_bytes, moe_positions, moe_replan, moe_route,
                      moe_slot_bytes, moe_slot_sections, moe_status_string, moe_swiglu_backward,
                      moe_test_mfma_loop, moe_test_mxfp4_probe, moe_test_stream_read,
                      moe_workspace_bytes)

binding.load()

__all__ = ["binding", "MOE_DT_BF16", "MOE_DT_FP16", "MOE_DT_FP32", "MOE_OP_DEMAND", "MOE_OP_EXPERTS", "MOE_OP_HOT_PICK", "MOE_OP_ROUTE",
           "MoeError", "arena_load_slot", "check", "moe_combine",
           "moe_combine_backward", "moe_demand_accumulate", "moe_dispatch",
           "moe_dispatch_backward", "moe_int8_matmul", "moe_int8_quantize", "moe_int8_row_bytes",
           "moe_positions", "moe_grouped_matmul", "moe_grouped_outer", "moe_grouped_outer_ws_bytes",
           "moe_swiglu_backward",
           "moe_int4_code_bytes", "moe_int4_scale_count", "moe_int4_quantize", "moe_int4_matmul",
           "moe_experts_forward", "moe_hot_install", "moe_hot_pick", "moe_mxfp4_row_bytes", "moe_replan", "moe_route", "moe_slot_bytes",
           "moe_slot_sections", "moe_status_string", "moe_test_mfma_loop", "moe_test_mxfp4_probe",
           "moe_test_stream_read", "moe_workspace_bytes"]
