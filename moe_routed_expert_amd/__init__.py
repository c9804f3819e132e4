"""MI355X-native routed-expert epilogue: clamped SwiGLU x routing probability and the
fp32 router-weight multiply, each with a forward and a single-pass backward, and the
gate_up grouped GEMM with the clamped SwiGLU epilogue fused into it (bf16 MFMA),
the down-projection grouped GEMM with the router-weight multiply fused into it,
and the fp32 combine of routed rows into tokens, as hand-written HIP kernels for
gfx950 behind a C ABI (include/moe_epi.h); and the steps around the experts
(include/moe_routed.h): the order of the routed rows, the dispatch of tokens and the
weighted combine with their gradients, and the experts' products in 8-bit integers; and
the steps before them (include/moe_prologue.h): the norm that joins the residual stream, the
router's product and the choice of each token's experts, with their gradients.

The binding loads libmoe_epi.so on first use and raises if it is not built.
"""
from .binding import (MoeEpiError, RouterWeightMul, SwigluClamped, grouped_down_router_fwd,
                      grouped_gate_up_swiglu_fwd, moe_combine_fwd, router_weight_mul,
                      router_weight_mul_bwd, router_weight_mul_fwd, swiglu_clamped,
                      swiglu_clamped_bwd, swiglu_clamped_fwd)
from .prologue import (MoeRoute, MoeRouterLogits, RmsNorm, moe_route, moe_route_bwd, moe_route_fwd, moe_router_logits,
                       moe_router_logits_bwd, moe_router_logits_bwd_workspace_bytes, moe_router_logits_fwd,
                       moe_router_logits_workspace_bytes, rms_norm, rms_norm_bwd, rms_norm_bwd_workspace_bytes,
                       rms_norm_fwd, rms_norm_int8)
from .routed import (MoeCombineWeighted, MoeDispatch, grouped_down_router_int8_fwd,
                     grouped_gate_up_swiglu_int8_fwd, moe_combine_weighted_bwd, moe_combine_weighted_fwd,
                     moe_dispatch_bwd, moe_dispatch_fwd, moe_sort, moe_sort_fwd, moe_sort_workspace_bytes,
                     quantize_rows_int8, quantize_rows_int8_fwd)

__all__ = [
    "MoeEpiError", "RouterWeightMul", "SwigluClamped", "grouped_down_router_fwd", "grouped_gate_up_swiglu_fwd",
    "moe_combine_fwd", "router_weight_mul",
    "router_weight_mul_bwd",
    "router_weight_mul_fwd", "swiglu_clamped", "swiglu_clamped_bwd", "swiglu_clamped_fwd",
    "MoeCombineWeighted", "MoeDispatch", "grouped_down_router_int8_fwd", "grouped_gate_up_swiglu_int8_fwd",
    "moe_combine_weighted_bwd", "moe_combine_weighted_fwd", "moe_dispatch_bwd", "moe_dispatch_fwd", "moe_sort",
    "moe_sort_fwd", "moe_sort_workspace_bytes", "quantize_rows_int8", "quantize_rows_int8_fwd",
    "MoeRoute", "MoeRouterLogits", "RmsNorm", "moe_route", "moe_route_bwd", "moe_route_fwd", "moe_router_logits",
    "moe_router_logits_bwd", "moe_router_logits_bwd_workspace_bytes", "moe_router_logits_fwd",
    "moe_router_logits_workspace_bytes", "rms_norm", "rms_norm_bwd", "rms_norm_bwd_workspace_bytes", "rms_norm_fwd",
    "rms_norm_int8",
]
