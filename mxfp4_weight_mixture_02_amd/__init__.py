"""MI355X (gfx950) MXFP4 mixture-of-experts expert block.

The work runs in libmxfp4_moe.so (C ABI in include/mxfp4_moe.h); this
package only marshals torch tensors into it.
"""
from .native import (Dims, MoeLayer, Mxfp4Error, SavedState, Workspace, lib,  # noqa: F401
                     mxfp4_dequantize, mxfp4_moe_backward, mxfp4_moe_backward_dx, mxfp4_moe_forward,
                     mxfp4_moe_forward_noalloc, mxfp4_quantize, mxfp8_quantize,
                     workspace_bytes)
from .ops import (BalanceLoss, Fp4Matrix, Fp8Matrix, Normed, RouteOptions, Routing, SavedState8,  # noqa: F401
                  SwigluCheckpoint, fp4_linear, fp4_linear_dx, fp4_matmul, fp4_matrix, fp4_quantize, fp8_linear,
                  fp8_linear_dw, fp8_linear_dx, fp8_matmul, fp8_quantize, fp8_quantize_t, fp8_transpose, moe_balance,
                  moe_balance_backward, moe_route, moe_route_backward, moe_router_logits,
                  mxfp4_moe_backward_routed, mxfp4_moe_forward_routed, rms_norm, rms_norm_backward, swiglu_mxfp8,
                  swiglu_mxfp8_backward, swiglu_mxfp8_restore)
