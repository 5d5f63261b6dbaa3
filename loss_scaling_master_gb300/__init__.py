"""GB300-native mixed-precision optimizer step: loss-scale unscale/check,
dynamic scale state machine, FP32-master AdamW with bf16 emission, and
tensorwise dynamic FP8 quantization with transposed copies; and the operators
around it in the forward and backward pass: microscaled 4-bit quantisation,
products and linear layers, layer norm, activations kept in 8 bits, dropout, log
probabilities of tokens.

The compute lives in libampfp8.so (hand-written CUDA for sm_103a, C ABI in
include/ampfp8.h and include/ampops.h); this package is its thin binding.
"""
from ._lib import (AmpError, TensorList, amp_abi_version, amp_adamw_master_step,
                   amp_adamw_master_step_clip, amp_adamw_master_step_fp8_delayed,
                   amp_adamw_master_step_sr, amp_emit_bf16, amp_selftest_bounded_wait,
                   amp_adamw_master_step_clip_sr, amp_adamw_master_step_fp8_delayed_sr,
                   fp8_quant_tensorwise_list_sr, amp_tensor_list_check,
                   amp_noalloc_check, amp_tensor_list_copy_from_host,
                   amp_tensor_list_copy_to_host, amp_read_state, amp_scale_health, ScalerState,
                   fp8_quant_groupwise,
                   amp_adamw_master_step_noalloc, amp_last_error, amp_update_scale_fp8_history,
                   amp_unscale_check_norm, amp_tensor_list_create, amp_tensor_list_destroy,
                   amp_tensor_list_set_amax_slots, amp_unscale_check, amp_update_scale,
                   fp8_quant_rowwise, fp8_quant_tensorwise, fp8_quant_tensorwise_list, load)
from . import ops
from .ops import (amp_act_backward_mx8, amp_act_forward_mx8, amp_bias_act_backward_mx8,
                  amp_ckpt8_restore, amp_ckpt8_save, amp_dropout_backward, amp_dropout_forward,
                  amp_token_logprobs_backward, amp_token_logprobs_forward, fp4_linear_mx,
                  amp_layer_norm_backward, amp_layer_norm_forward, amp_layer_norm_workspace,
                  ckpt8_buffers, fp4_dequant_mx, fp4_mx_buffers, fp4_mx_check, fp4_product_mx,
                  fp4_quant_mx)
from .step import AmpOptimizerStep

__all__ = ["AmpError", "TensorList", "AmpOptimizerStep", "load", "amp_abi_version",
           "amp_last_error", "amp_tensor_list_create", "amp_tensor_list_destroy",
           "amp_tensor_list_set_amax_slots", "amp_unscale_check", "amp_adamw_master_step",
           "amp_adamw_master_step_noalloc", "amp_adamw_master_step_clip", "amp_emit_bf16",
           "amp_unscale_check_norm", "amp_adamw_master_step_fp8_delayed",
           "amp_adamw_master_step_sr", "amp_tensor_list_check", "amp_selftest_bounded_wait", "amp_noalloc_check",
           "amp_tensor_list_copy_from_host", "amp_tensor_list_copy_to_host", "amp_read_state",
           "amp_scale_health", "ScalerState", "fp8_quant_groupwise",
           "amp_update_scale_fp8_history",
           "fp8_quant_tensorwise", "fp8_quant_tensorwise_list", "fp8_quant_rowwise",
           "amp_update_scale", "amp_adamw_master_step_clip_sr",
           "amp_adamw_master_step_fp8_delayed_sr", "fp8_quant_tensorwise_list_sr",
           "fp4_quant_mx", "fp4_dequant_mx", "fp4_product_mx", "fp4_mx_buffers", "fp4_mx_check",
           "amp_layer_norm_forward", "amp_layer_norm_backward", "amp_layer_norm_workspace",
           "amp_act_forward_mx8", "amp_act_backward_mx8", "amp_ckpt8_save", "amp_ckpt8_restore",
           "ckpt8_buffers", "fp4_linear_mx", "amp_bias_act_backward_mx8", "amp_dropout_forward",
           "amp_dropout_backward", "amp_token_logprobs_forward", "amp_token_logprobs_backward"]
