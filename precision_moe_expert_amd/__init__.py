"""MI355X (gfx950) low-precision MoE expert forward.

The compute lives in libmoe_lp.so (HIP kernels behind the C ABI of
include/moe_lp.h); `binding` marshals torch tensors into it.  `synth` holds the
seeded synthetic input generators.
"""
from . import binding  # noqa: F401
from .binding import (FMT_FP8, FMT_FP8_POW2, FMT_INT4, FMT_MXFP4, FMT_NVFP4, GATE_SIGMOID, GATE_SOFTMAX,  # noqa: F401
                      GROUP_MAX, GROUP_TOP2, LINEAR_D_W, LINEAR_D_X, LINEAR_FORWARD, WL_KBLOCKED, WL_ROWS,
                      MoeError, balance_loss, balance_loss_backward, clip_grads, combine, expert_backward,
                      expert_backward_gated, expert_forward, expert_forward_gated, expert_forward_materialized,
                      expert_forward_noalloc, fp8_linear, fp8_linear_backward, fp8_linear_transpose,
                      fp8_linear_workspace_bytes, grad_norm, lm_head_distill, lm_head_distill_backward,
                      lm_head_logprob, lm_head_loss, lm_head_loss_backward, make_gate, make_layer,
                      pack_weights_kblocked, prepare_backward_weights, route_gated, route_gated_backward,
                      route_permute, scale_grads, workspace_bytes)
