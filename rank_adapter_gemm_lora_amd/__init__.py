"""MI355X-native multi-adapter LoRA apply.

The compute lives in a C-ABI HIP library (include/lora.h, sources in csrc/);
:mod:`.binding` marshals arguments into it (same function names), and
:mod:`.synth` draws seeded synthetic workloads.  PyTorch, where callers use
it, only provides device memory and streams.
"""
from .binding import (EXPORTS, LORA_BF16, LORA_F32, LORA_MX_E2M1, LORA_MX_E4M3,  # noqa: F401
                      LoraError, lora_add_expand,
                      lora_add_shrink, lora_apply, lora_build_apply, lora_build_segments,
                      lora_build_shrink,
                      lora_evict_slot,
                      lora_get_device_status, lora_load_slot, lora_segments_create,
                      lora_segments_destroy, lora_segments_download, lora_segments_set_dense_min,
                      lora_segments_tile_counts, lora_slot_info, lora_merge_slot, lora_stack_create,
                      lora_stack_destroy, lora_status_string, lora_residency_create,
                      lora_residency_destroy, lora_residency_register, lora_residency_unregister,
                      lora_residency_map_batch, lora_residency_slot_of, lora_residency_stats,
                      lora_mx_code_bytes, lora_mx_scale_bytes, lora_mx_quantize,
                      lora_mx_dequantize, lora_mx_weight_create, lora_mx_weight_destroy,
                      lora_mx_weight_load, lora_mx_weight_load_packed, lora_mx_linear,
                      lora_rmsnorm_mx, lora_swiglu_mx, lora_block_norm_mx,
                      LORA_ACT_NONE, LORA_ACT_RELU, LORA_ACT_SILU, LORA_ACT_GELU,
                      LORA_ACT_GELU_TANH, LORA_ACT_SWIGLU, lora_mx_linear_fused,
                      LORA_MOE_SIGMOID, LORA_MOE_SOFTMAX, lora_moe_plan_create,
                      lora_moe_plan_destroy, lora_moe_route, lora_moe_group, lora_moe_combine,
                      LORA_MOE_PAIRS, LORA_MOE_ROWS, lora_mx_experts_create,
                      lora_mx_experts_destroy, lora_mx_experts_load,
                      lora_mx_experts_load_packed, lora_mx_expert_linear)
