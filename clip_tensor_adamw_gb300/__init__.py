"""clip + AdamW optimizer step on one GB300 (sm_103a): ScaleTensors, ClipGradNorms and AdamWSteps (also over
parameter groups, and both as one fused step), ClipGradNorms fused into the gradients' last write when that write is
an add, and SGD / SGD with momentum over the same lists; the step whose update is orthogonalised by Newton-Schulz products
(muon.py); and, before the step, losses over logits and from hidden states with their gradients, and activation checkpoints
in 8 bits with the backward passes that read them (train.py).

The compute lives in libmica_optim.so (hand-written CUDA kernels behind the C ABI of include/mica_optim.h); this
package is its Python binding. Build the library with ``python -m clip_tensor_adamw_gb300.build``.
"""
from .mica import (GroupIndex, MicaError, TensorList, lib, mica_accumulate_clip_grad_norms,
                   mica_accumulate_grad_sumsq, mica_adamw_steps,
                   mica_adamw_steps_grouped, mica_clip_adamw_step, mica_clip_factor_from_sumsq, mica_clip_grad_norms, mica_grad_sumsq,
                   mica_launch_count, mica_release_cache,
                   mica_scale_tensors, mica_selftest_grid_wait_timeout, mica_selftest_wait_timeout, mica_sgd_steps,
                   mica_sync, mica_work_items)
from .muon import mica_muon_steps, mica_orthogonalize
from .train import (LinearCrossEntropy, PackedActivation, PolicyLoss, PreferenceLoss, mica_act_grad, mica_act_pack,
                    mica_act_unpack, mica_linear_cross_entropy, mica_linear_logps, mica_linear_logps_grad,
                    mica_packed_wgrad, mica_policy_loss, mica_preference_loss, mica_token_logps, mica_token_logps_grad)

__all__ = ["GroupIndex", "MicaError", "TensorList", "lib", "mica_accumulate_clip_grad_norms",
           "mica_accumulate_grad_sumsq", "mica_adamw_steps",
           "mica_adamw_steps_grouped",
           "mica_clip_adamw_step", "mica_clip_factor_from_sumsq", "mica_clip_grad_norms", "mica_grad_sumsq",
           "mica_launch_count", "mica_release_cache",
           "mica_scale_tensors", "mica_selftest_grid_wait_timeout", "mica_selftest_wait_timeout", "mica_sgd_steps",
           "mica_sync", "mica_work_items",
           "PackedActivation", "PolicyLoss", "PreferenceLoss", "mica_act_grad", "mica_act_pack", "mica_act_unpack",
           "mica_muon_steps", "mica_orthogonalize", "LinearCrossEntropy", "mica_linear_cross_entropy", "mica_linear_logps", "mica_linear_logps_grad",
           "mica_packed_wgrad", "mica_policy_loss", "mica_preference_loss", "mica_token_logps", "mica_token_logps_grad"]
