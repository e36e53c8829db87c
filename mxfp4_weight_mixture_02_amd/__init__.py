"""MI355X (gfx950) MXFP4 mixture-of-experts expert block.

The work runs in libmxfp4_moe.so (C ABI in include/mxfp4_moe.h); this
package only marshals torch tensors into it.
"""
from .native import (Dims, MoeLayer, Mxfp4Error, SavedState, Workspace, lib,  # noqa: F401
                     mxfp4_dequantize, mxfp4_moe_backward, mxfp4_moe_backward_dx, mxfp4_moe_forward,
                     mxfp4_moe_forward_noalloc, mxfp4_quantize, mxfp8_quantize,
                     workspace_bytes)
from .ops import (Fp8Matrix, RouteOptions, Routing, SavedState8, SwigluCheckpoint,  # noqa: F401
                  fp8_linear, fp8_linear_dw, fp8_linear_dx, fp8_matmul, fp8_quantize, fp8_quantize_t,
                  fp8_transpose, moe_route, moe_route_backward, moe_router_logits,
                  mxfp4_moe_backward_routed, mxfp4_moe_forward_routed, swiglu_mxfp8,
                  swiglu_mxfp8_backward, swiglu_mxfp8_restore)
