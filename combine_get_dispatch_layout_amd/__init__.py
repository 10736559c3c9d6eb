"""MI355X-native MoE expert-parallel token shuffle: routing layout, slot
assignment, dispatch (optionally FP8 E4M3FN / int8 quantised) and weighted
combine, with the router and its balance loss, products with bf16, 4-bit and
int8 expert weights and the whole expert layer for a few tokens beside them, as
hand-written HIP kernels for gfx950 behind a C ABI (include/ep.h, include/ep_moe.h).  This package holds the
kernels (csrc/), their build script and the thin Python binding (ep.py,
moe.py)."""
from .ep import (Config, EpError, Handle, ep_check_error, ep_combine, ep_dispatch,  # noqa: F401
                 ep_get_layout, ep_handle_free, ep_handle_get_view, ep_handle_init,
                 ep_layout_dispatch, ep_quantize_rows, ep_dispatch_topk, ep_dispatch_overlap,
                 ep_combine_overlap,
                 ep_recv_capacity, ep_workspace_size, EP_QUANT_NONE, EP_QUANT_FP8_E4M3,
                 EP_QUANT_INT8, EP_QUANT_MXFP4, EP_SCALE_FP32, EP_SCALE_POW2, EP_SCALE_UE8M0)
from .moe import (Balance, BalanceConfig, GateConfig, Weights, ep_balance_loss,  # noqa: F401
                  ep_balance_loss_backward, ep_balance_workspace_size, ep_expert_matmul,
                  ep_expert_matvec, ep_gate, ep_gate_backward, ep_matmul,
                  ep_matmul_workspace_size, ep_matvec, ep_moe_layer,
                  ep_moe_workspace_size, EP_ACT_NONE, EP_ACT_SWIGLU, EP_SCORE_SIGMOID,
                  EP_SCORE_SOFTMAX, EP_WEIGHT_BF16, EP_WEIGHT_INT4, EP_WEIGHT_INT8,
                  EP_WEIGHT_MXFP4)
