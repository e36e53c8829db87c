"""ctypes binding of the operators in include/mxmoe_ops.h: routing with its
gradient, dense products in 8-bit floating point and 8-bit activation
checkpoints.

Argument marshalling only, as in native.py.  Each call runs on its tensors'
device and that device's current stream, whatever device is current; scratch
is allocated for the call on that stream, so calls on several streams, and
several captured graphs, share nothing.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import native
from .native import Dims, Grads, MoeLayer, Mxfp4Error, Saved, SavedState, Weights

SCORES = {"softmax": 0, "sigmoid": 1}
GROUP_SCORES = {"max": 0, "top2": 1}


class _RouteOpts(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("groups", ctypes.c_int32), ("top_groups", ctypes.c_int32),
                ("group_score", ctypes.c_int32), ("renorm", ctypes.c_int32), ("scale", ctypes.c_float)]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library with the operators' signatures declared."""
    global _lib
    if _lib is None:
        L = native.lib()
        vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
        opts = ctypes.POINTER(_RouteOpts)
        L.mxmoe_route_workspace_bytes.restype = sz
        L.mxmoe_route_workspace_bytes.argtypes = [i64, i32, i32]
        L.mxmoe_route.argtypes = [opts, i64, i32, i32] + [vp] * 7 + [sz, vp]
        L.mxmoe_route_backward.argtypes = [opts, i64, i32, i32] + [vp] * 5
        ci, f32 = ctypes.c_int, ctypes.c_float
        for n, more in (("matmul", [ci]), ("linear", [ci]), ("linear_dw", [])):
            f = getattr(L, f"mxmoe_fp8_{n}_workspace_bytes")
            f.restype, f.argtypes = sz, [i64, i64, i64] + more
        L.mxmoe_fp8_quantize.argtypes = [vp, ci, i64, i64, ci, vp, vp, vp]
        L.mxmoe_fp8_quantize_t.argtypes = [vp, ci, i64, i64, vp, vp, vp]
        L.mxmoe_fp8_transpose.argtypes = [vp, vp, i64, i64, vp, vp, vp]
        L.mxmoe_fp8_matmul.argtypes = [i64, i64, i64, vp, vp, vp, vp, ci, vp, ci, vp, vp, sz, vp]
        L.mxmoe_fp8_linear.argtypes = [i64, i64, i64, vp, vp, vp, vp, ci, vp, vp, sz, vp]
        L.mxmoe_fp8_linear_dw.argtypes = [i64, i64, i64, vp, vp, vp, vp, sz, vp]
        layer = [ctypes.POINTER(Dims), ctypes.POINTER(Weights)]
        L.mxmoe_router_logits.argtypes = [i64, i64, i32] + [vp] * 5
        L.mxmoe_forward_routed.argtypes = layer + [vp, vp, ctypes.POINTER(Saved), vp, sz, vp]
        L.mxmoe_backward_routed.argtypes = layer + [ctypes.POINTER(Saved), vp, vp, ctypes.POINTER(Grads),
                                                    vp, vp, sz, vp]
        L.mxmoe_swiglu8_forward.argtypes = [vp, i64, i64, f32, f32, vp, vp, vp, vp]
        L.mxmoe_swiglu8_backward.argtypes = [vp, vp, vp, i64, i64, f32, f32, vp, vp, vp]
        L.mxmoe_swiglu8_restore.argtypes = [vp, vp, i64, i64, f32, f32, vp, vp, vp]
        for n in ("route", "route_backward", "router_logits", "forward_routed", "backward_routed", "fp8_quantize",
                  "fp8_quantize_t", "fp8_transpose", "fp8_matmul", "fp8_linear", "fp8_linear_dw",
                  "swiglu8_forward", "swiglu8_backward", "swiglu8_restore"):
            getattr(L, "mxmoe_" + n).restype = ci
        _lib = L
    return _lib


def _shape(t, shape, dtype, name, optional=False):
    """Refuse a tensor whose shape or dtype differs from what the C ABI will
    assume; before the device checks, and on any device."""
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is required")
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")


def _same_device(**tensors):
    """Every tensor contiguous and on one GPU; returns that device."""
    dev = None
    for name, t in tensors.items():
        if t is None:
            continue
        if not (t.is_cuda and t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"{name} is on {t.device}, other tensors on {dev}")
    return dev


_functions = {}


def _function(name):
    f = _functions.get(name)
    if f is None:
        f = _functions[name] = getattr(lib(), name)
    return f


def _call(name, dev, *args):
    """<name>(*args, stream) on dev and its current stream."""
    fn, index = _function(name), dev.index
    if torch.cuda.current_device() == index:
        rc = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if rc != native.MXFP4_OK:
        raise Mxfp4Error(name, rc, lib().mxfp4_last_error().decode())


def _p(t):
    return None if t is None else t.data_ptr()


def _bytes_needed(name, *args):
    n = _function(name)(*args)
    if n == 0:
        raise Mxfp4Error(name, -1, lib().mxfp4_last_error().decode())
    return n


_unused = {}


def _workspace(name, dev, *args):
    """(scratch for the call, its bytes).  Up to 256 bytes are never used (a
    call that needs no scratch asks for them), so one tensor serves all."""
    n = _bytes_needed(name, *args)
    if n > 256:
        return torch.empty(n, dtype=torch.uint8, device=dev), n
    t = _unused.get(dev)
    if t is None:
        t = torch.empty(256, dtype=torch.uint8, device=dev)
        if not torch.cuda.is_current_stream_capturing():   # a graph's memory is the graph's
            _unused[dev] = t
    return t, n


# ---------------------------------------------------------------- routing

@dataclass(frozen=True)
class RouteOptions:
    """How logits become a routing (mxmoe_route_opts)."""
    score: str = "softmax"        # softmax | sigmoid
    groups: int = 1               # groups of consecutive experts
    top_groups: int = 1           # groups whose experts may be chosen
    group_score: str = "max"      # max | top2: a group's value
    renorm: bool = True           # weights divided by the chosen scores' sum
    scale: float = 1.0

    def __post_init__(self):
        if self.score not in SCORES:
            raise ValueError(f"score must be one of {sorted(SCORES)}")
        if self.group_score not in GROUP_SCORES:
            raise ValueError(f"group_score must be one of {sorted(GROUP_SCORES)}")
        object.__setattr__(self, "struct", _RouteOpts(
            SCORES[self.score], self.groups, self.top_groups, GROUP_SCORES[self.group_score],
            int(self.renorm), self.scale))


@dataclass
class Routing:
    """A routing of T tokens as the expert block takes it."""
    topk_idx: torch.Tensor        # int32 [T, k], descending choice value
    topk_w: torch.Tensor          # fp32 [T, k]
    expert_offsets: torch.Tensor  # int32 [E + 1]
    sorted_rows: torch.Tensor     # int32 [T*k]


def _logits(logits):
    if logits.dim() != 2:
        raise ValueError(f"logits must be [T, E], got {tuple(logits.shape)}")
    T, E = logits.shape
    _shape(logits, (T, E), torch.float32, "logits")
    return T, E


def moe_route(logits: torch.Tensor, k: int, options: RouteOptions = RouteOptions(),
              bias: torch.Tensor | None = None) -> Routing:
    """Routing from fp32 logits [T, E]: scores, the choice on score + bias
    (within the best groups), weights and the permutation plan."""
    T, E = _logits(logits)
    _shape(bias, (E,), torch.float32, "bias", optional=True)
    dev = _same_device(logits=logits, bias=bias)
    ws, nbytes = _workspace("mxmoe_route_workspace_bytes", dev, T, E, k)
    # one allocation for the four: they are most of a small call's time (1.6 us each)
    R = T * k
    idx, w, rows, off = torch.unsafe_split_with_sizes(
        torch.empty(3 * R + E + 1, dtype=torch.int32, device=dev), (R, R, R, E + 1))
    r = Routing(idx.view(T, k), w.view(torch.float32).view(T, k), off, rows)
    _call("mxmoe_route", dev, options.struct, T, E, k, _p(logits), _p(bias), _p(r.topk_idx),
          _p(r.topk_w), _p(r.expert_offsets), _p(r.sorted_rows), _p(ws), nbytes)
    return r


def moe_route_backward(logits: torch.Tensor, topk_idx: torch.Tensor, dw: torch.Tensor,
                       options: RouteOptions = RouteOptions()) -> torch.Tensor:
    """dlogits fp32 [T, E] from dw [T, k], the gradient of the routing
    weights, with the choice held fixed."""
    T, E = _logits(logits)
    if topk_idx.dim() != 2:
        raise ValueError(f"topk_idx must be [T, k], got {tuple(topk_idx.shape)}")
    k = topk_idx.shape[1]
    _shape(topk_idx, (T, k), torch.int32, "topk_idx")
    _shape(dw, (T, k), torch.float32, "dw")
    dev = _same_device(logits=logits, topk_idx=topk_idx, dw=dw)
    out = torch.empty_like(logits)
    _call("mxmoe_route_backward", dev, options.struct, T, E, k, _p(logits), _p(topk_idx), _p(dw),
          _p(out))
    return out


def moe_router_logits(layer: MoeLayer, x: torch.Tensor) -> torch.Tensor:
    """The layer's router logits fp32 [T, E] of bf16 x [T, H]: fp64 sums,
    rounded once (the values mxfp4_moe_forward routes by)."""
    layer.check_shapes()
    if x.dim() != 2:
        raise ValueError(f"x must be [T, H], got {tuple(x.shape)}")
    T = x.shape[0]
    _shape(x, (T, layer.H), torch.bfloat16, "x")
    dev = _same_device(x=x, router_w=layer.router_w, router_b=layer.router_b)
    out = torch.empty((T, layer.E), dtype=torch.float32, device=dev)
    _call("mxmoe_router_logits", dev, T, layer.H, layer.E, _p(x), _p(layer.router_w), _p(layer.router_b), _p(out))
    return out


def _layer_device(layer, **tensors):
    names = ("gu_codes", "gu_scales", "gu_bias", "dn_codes", "dn_scales", "dn_bias", "lora_A", "lora_B",
             "lora_gu_A", "lora_gu_B")
    return _same_device(**tensors, **{n: getattr(layer, n) for n in names})


def _routing_shapes(layer, T, r):
    _shape(r.topk_idx, (T, layer.k), torch.int32, "topk_idx")
    _shape(r.topk_w, (T, layer.k), torch.float32, "topk_w")
    _shape(r.expert_offsets, (layer.E + 1,), torch.int32, "expert_offsets")
    _shape(r.sorted_rows, (T * layer.k,), torch.int32, "sorted_rows")


def _fields(r):
    return dict(topk_idx=r.topk_idx, topk_w=r.topk_w, expert_offsets=r.expert_offsets, sorted_rows=r.sorted_rows)


def mxfp4_moe_forward_routed(layer: MoeLayer, x: torch.Tensor, routing: Routing, saved: bool | str = False):
    """The expert block on a given routing (moe_route of the same T, E and
    k).  Returns (out, state): state None, or with ``saved`` True a
    SavedState, with "mxfp8" a SavedState8, that holds the routing's tensors
    and the activations."""
    layer.check_shapes(routed=True)
    if x.dim() != 2:
        raise ValueError(f"x must be [T, H], got {tuple(x.shape)}")
    T = x.shape[0]
    _shape(x, (T, layer.H), torch.bfloat16, "x")
    _routing_shapes(layer, T, routing)
    if not isinstance(saved, bool):
        SavedState8.check_format(saved)
    dev = _layer_device(layer, x=x, **_fields(routing))
    state = SavedState(**_fields(routing), h=None, a=None)
    if saved:
        full = SavedState.empty(layer, T, dev)
        state.h, state.a, state.lora_v, state.lora_vg = full.h, full.a, full.lora_v, full.lora_vg
    nbytes = native.workspace_bytes(layer, T, native.WS_FORWARD_SAVED if saved else native.WS_FORWARD)
    out = torch.empty_like(x)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    _call("mxmoe_forward_routed", dev, layer.dims(T), layer.weights(routed=True), _p(x), _p(out), state.struct(),
          _p(ws), nbytes)
    if isinstance(saved, str):
        state = SavedState8.pack(layer, state)
    return out, state if saved else None


def mxfp4_moe_backward_routed(layer: MoeLayer, saved, dy: torch.Tensor, x: torch.Tensor | None = None,
                              base: bool = False) -> dict:
    """The backward of mxfp4_moe_forward_routed from its SavedState or
    SavedState8: dx (no router term), dw [T, k] (the routing weights'
    gradient, moe_route_backward's input), the adapter gradients the layer
    has, and with ``base`` the base-weight and bias gradients.  ``x``, the
    forward's input, is needed with ``base`` or a gate_up adapter."""
    layer.check_shapes(routed=True)
    if dy.dim() != 2:
        raise ValueError(f"dy must be [T, H], got {tuple(dy.shape)}")
    T = dy.shape[0]
    E, H, I = layer.E, layer.H, layer.I
    _shape(dy, (T, H), torch.bfloat16, "dy")
    _shape(x, (T, H), torch.bfloat16, "x", optional=not base and layer.lora_gu_A is None)
    saved.check_shapes(layer, T)
    saved = native._restored(saved)
    dev = _layer_device(layer, dy=dy, x=x, h=saved.h, a=saved.a, lora_v=saved.lora_v, lora_vg=saved.lora_vg,
                        **_fields(saved))
    f32 = dict(dtype=torch.float32, device=dev)
    out = {"dx": torch.empty_like(dy), "dw": torch.empty((T, layer.k), **f32)}
    for name, t in (("dA", layer.lora_A), ("dB", layer.lora_B), ("dA_gu", layer.lora_gu_A),
                    ("dB_gu", layer.lora_gu_B)):
        if t is not None:
            out[name] = torch.empty(t.shape, **f32)
    if base:
        out.update(dW_gu=torch.empty((E, 2 * I, H), **f32), dW_dn=torch.empty((E, H, I), **f32),
                   db_gu=torch.empty((E, 2 * I), **f32), db_dn=torch.empty((E, H), **f32))
    nbytes = native.workspace_bytes(layer, T, native.WS_BACKWARD_FULL if base else native.WS_BACKWARD)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    grads = Grads(*[_p(out.get(n)) for n, _ in Grads._fields_])
    _call("mxmoe_backward_routed", dev, layer.dims(T), layer.weights(routed=True), saved.struct(), _p(x), _p(dy),
          grads, _p(out["dw"]), _p(ws), nbytes)
    return out


# ------------------------------------------------------ 8-bit dense products

_DTYPES = {torch.float32: 0, torch.bfloat16: 1}


def _up(n, m):
    return (n + m - 1) // m * m


@dataclass
class Fp8Matrix:
    """A [rows, K] matrix in 8-bit floating point (E4M3) with one power-of-two
    scale for each block of block_rows x 128 (layouts in mxmoe_ops.h)."""
    codes: torch.Tensor      # uint8 [rows, K rounded up to 128], zeros past K
    scales: torch.Tensor     # uint8 [K blocks, rows rounded up to 16 | row blocks of 128]
    K: int
    block_rows: int          # 1 or 128

    @property
    def rows(self):
        return self.codes.shape[0]

    @staticmethod
    def empty(rows, K, block_rows, device):
        if block_rows not in (1, 128):
            raise ValueError(f"block_rows must be 1 or 128, got {block_rows}")
        if rows < 1 or K < 1:
            raise ValueError(f"an 8-bit matrix has at least one element, got {rows} x {K}")
        Kp = _up(K, 128)
        side = _up(rows, 16) if block_rows == 1 else _up(rows, 128) // 128
        u8 = dict(dtype=torch.uint8, device=device)
        return Fp8Matrix(torch.empty((rows, Kp), **u8), torch.empty((Kp // 128, side), **u8), K, block_rows)

    def check_shapes(self, name="matrix"):
        if self.codes.dim() != 2 or self.block_rows not in (1, 128) or self.K < 1:
            raise ValueError(f"{name}: codes must be [rows, K rounded up to 128], block_rows 1 or 128")
        Kp = _up(self.K, 128)
        side = _up(self.rows, 16) if self.block_rows == 1 else _up(self.rows, 128) // 128
        _shape(self.codes, (self.rows, Kp), torch.uint8, name + ".codes")
        _shape(self.scales, (Kp // 128, side), torch.uint8, name + ".scales")


def _matrix(x, name):
    if x.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got {tuple(x.shape)}")
    if x.dtype not in _DTYPES:
        raise ValueError(f"{name} must be fp32 or bf16, got {x.dtype}")
    return x.shape


def fp8_quantize(x: torch.Tensor, block_rows: int = 1) -> Fp8Matrix:
    """fp32 or bf16 x [rows, K] in blocks of block_rows x 128."""
    rows, K = _matrix(x, "x")
    dev = _same_device(x=x)
    q = Fp8Matrix.empty(rows, K, block_rows, dev)
    _call("mxmoe_fp8_quantize", dev, _p(x), _DTYPES[x.dtype], rows, K, block_rows, _p(q.codes), _p(q.scales))
    return q


def fp8_quantize_t(x: torch.Tensor) -> Fp8Matrix:
    """x's transpose [K, rows] in blocks of 128 of x's rows, one column each."""
    rows, K = _matrix(x, "x")
    dev = _same_device(x=x)
    q = Fp8Matrix.empty(K, rows, 1, dev)
    _call("mxmoe_fp8_quantize_t", dev, _p(x), _DTYPES[x.dtype], rows, K, _p(q.codes), _p(q.scales))
    return q


def fp8_transpose(w: Fp8Matrix) -> Fp8Matrix:
    """The transpose of a matrix with 128 x 128 blocks, exactly."""
    w.check_shapes("w")
    if w.block_rows != 128:
        raise ValueError("only a matrix with block_rows 128 can be transposed exactly")
    dev = _same_device(codes=w.codes, scales=w.scales)
    t = Fp8Matrix.empty(w.K, w.rows, 128, dev)
    _call("mxmoe_fp8_transpose", dev, _p(w.codes), _p(w.scales), w.rows, w.K, _p(t.codes), _p(t.scales))
    return t


def _out(M, N, dtype, dev):
    if dtype not in _DTYPES:
        raise ValueError(f"dtype must be fp32 or bf16, got {dtype}")
    return torch.empty((M, N), dtype=dtype, device=dev)


def fp8_matmul(x: Fp8Matrix, w: Fp8Matrix, bias: torch.Tensor | None = None,
               dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """x [M, K] (block_rows 1) times w [N, K] (either block shape) transposed,
    plus bias bf16 [N]: [M, N] in dtype."""
    x.check_shapes("x")
    w.check_shapes("w")
    if x.block_rows != 1:
        raise ValueError("x needs block_rows 1")
    if x.K != w.K:
        raise ValueError(f"x has K={x.K}, w K={w.K}")
    M, N = x.rows, w.rows
    _shape(bias, (N,), torch.bfloat16, "bias", optional=True)
    dev = _same_device(x=x.codes, x_scales=x.scales, w=w.codes, w_scales=w.scales, bias=bias)
    out = _out(M, N, dtype, dev)
    ws, nbytes = _workspace("mxmoe_fp8_matmul_workspace_bytes", dev, M, N, x.K, _DTYPES[dtype])
    _call("mxmoe_fp8_matmul", dev, M, N, x.K, _p(x.codes), _p(x.scales), _p(w.codes), _p(w.scales),
          w.block_rows, _p(bias), _DTYPES[dtype], _p(out), _p(ws), nbytes)
    return out


def fp8_linear(x: torch.Tensor, w: Fp8Matrix, bias: torch.Tensor | None = None,
               dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """bf16 x [M, K] rounded to E4M3 with a scale for each 128 elements of a
    row, times w [N, K] (128 x 128 blocks) transposed, plus bias: [M, N]."""
    if x.dim() != 2:
        raise ValueError(f"x must be [M, K], got {tuple(x.shape)}")
    w.check_shapes("w")
    if w.block_rows != 128:
        raise ValueError("w needs block_rows 128")
    M, N, K = x.shape[0], w.rows, w.K
    _shape(x, (M, K), torch.bfloat16, "x")
    _shape(bias, (N,), torch.bfloat16, "bias", optional=True)
    dev = _same_device(x=x, w=w.codes, w_scales=w.scales, bias=bias)
    out = _out(M, N, dtype, dev)
    ws, nbytes = _workspace("mxmoe_fp8_linear_workspace_bytes", dev, M, N, K, _DTYPES[dtype])
    _call("mxmoe_fp8_linear", dev, M, N, K, _p(x), _p(w.codes), _p(w.scales), _p(bias), _DTYPES[dtype],
          _p(out), _p(ws), nbytes)
    return out


def fp8_linear_dx(dy: torch.Tensor, w_t: Fp8Matrix, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """The input's gradient of fp8_linear: bf16 dy [M, N], rounded as x is,
    times w, given transposed (w_t = fp8_transpose(w), [K, N])."""
    return fp8_linear(dy, w_t, dtype=dtype)


def fp8_linear_dw(dy: torch.Tensor, x: torch.Tensor) -> torch.Tensor:
    """The weights' gradient of a linear layer, fp32 [N, K] = dy^T x, with
    bf16 dy [M, N] and x [M, K] rounded in blocks of 128 tokens."""
    if dy.dim() != 2 or x.dim() != 2:
        raise ValueError(f"dy and x must be 2-D, got {tuple(dy.shape)} and {tuple(x.shape)}")
    (M, N), K = dy.shape, x.shape[1]
    _shape(dy, (M, N), torch.bfloat16, "dy")
    _shape(x, (M, K), torch.bfloat16, "x")
    dev = _same_device(dy=dy, x=x)
    ws, nbytes = _workspace("mxmoe_fp8_linear_dw_workspace_bytes", dev, M, N, K)
    dw = torch.empty((N, K), dtype=torch.float32, device=dev)
    _call("mxmoe_fp8_linear_dw", dev, M, N, K, _p(dy), _p(x), _p(dw), _p(ws), nbytes)
    return dw


# ------------------------------------------------- 8-bit activation checkpoints

@dataclass
class SwigluCheckpoint:
    """The clamped SwiGLU's input h [R, 2I] in MXFP8, and its constants."""
    codes: torch.Tensor      # uint8 [R, 2I]
    scales: torch.Tensor     # uint8 [R, 2I / 32]
    alpha: float = 1.702
    limit: float = 7.0

    def check_shapes(self):
        if self.codes.dim() != 2 or self.codes.shape[1] % 32:
            raise ValueError(f"codes must be [R, 2I], 2I a multiple of 32, got {tuple(self.codes.shape)}")
        R, C = self.codes.shape
        _shape(self.codes, (R, C), torch.uint8, "codes")
        _shape(self.scales, (R, C // 32), torch.uint8, "scales")
        return R, C // 2


def _swiglu_rows(h):
    if h.dim() != 2 or h.shape[1] % 32:
        raise ValueError(f"h must be [R, 2I], 2I a multiple of 32, got {tuple(h.shape)}")
    _shape(h, tuple(h.shape), torch.bfloat16, "h")
    return h.shape[0], h.shape[1] // 2


def swiglu_mxfp8(h: torch.Tensor, alpha: float = 1.702, limit: float = 7.0, activation: bool = True):
    """The clamped SwiGLU of bf16 rows h [R, 2I] (gates even, ups odd) and an
    8-bit checkpoint of h: (a bf16 [R, I], checkpoint).  With activation
    False, (None, checkpoint)."""
    R, I = _swiglu_rows(h)
    dev = _same_device(h=h)
    u8 = dict(dtype=torch.uint8, device=dev)
    c = SwigluCheckpoint(torch.empty((R, 2 * I), **u8), torch.empty((R, I // 16), **u8), alpha, limit)
    a = torch.empty((R, I), dtype=torch.bfloat16, device=dev) if activation else None
    _call("mxmoe_swiglu8_forward", dev, _p(h), R, I, alpha, limit, _p(a), _p(c.codes), _p(c.scales))
    return a, c


def swiglu_mxfp8_backward(saved: SwigluCheckpoint, da: torch.Tensor, activation: bool = True):
    """(dh bf16 [R, 2I], a): the derivative at the checkpoint's values times
    da bf16 [R, I], and their activation (None with activation False)."""
    R, I = saved.check_shapes()
    _shape(da, (R, I), torch.bfloat16, "da")
    dev = _same_device(codes=saved.codes, scales=saved.scales, da=da)
    dh = torch.empty((R, 2 * I), dtype=torch.bfloat16, device=dev)
    a = torch.empty((R, I), dtype=torch.bfloat16, device=dev) if activation else None
    _call("mxmoe_swiglu8_backward", dev, _p(saved.codes), _p(saved.scales), _p(da), R, I, saved.alpha,
          saved.limit, _p(dh), _p(a))
    return dh, a


def swiglu_mxfp8_restore(saved: SwigluCheckpoint):
    """(h bf16 [R, 2I], a bf16 [R, I]): the checkpoint's values and their
    activation."""
    R, I = saved.check_shapes()
    dev = _same_device(codes=saved.codes, scales=saved.scales)
    h = torch.empty((R, 2 * I), dtype=torch.bfloat16, device=dev)
    a = torch.empty((R, I), dtype=torch.bfloat16, device=dev)
    _call("mxmoe_swiglu8_restore", dev, _p(saved.codes), _p(saved.scales), R, I, saved.alpha, saved.limit,
          _p(h), _p(a))
    return h, a


@dataclass
class SavedState8:
    """A forward's saved state with the gate_up output in 8 bits and without
    the activation: 2.06 I bytes a routed row against 6 I.  The backward
    restores both in bf16 for the time of the call; its gradients are those
    at the rounded gate_up output, with the forward's clamp decisions."""
    topk_idx: torch.Tensor
    topk_w: torch.Tensor
    expert_offsets: torch.Tensor
    sorted_rows: torch.Tensor
    checkpoint: SwigluCheckpoint
    lora_v: torch.Tensor | None = None
    lora_vg: torch.Tensor | None = None

    @staticmethod
    def check_format(name):
        if name != "mxfp8":
            raise ValueError(f'saved must be True, False or "mxfp8", got {name!r}')

    @staticmethod
    def pack(layer: MoeLayer, saved: SavedState) -> "SavedState8":
        """The 8-bit form of a forward's SavedState."""
        _, c = swiglu_mxfp8(saved.h, layer.alpha, layer.limit, activation=False)
        return SavedState8(**_fields(saved), checkpoint=c, lora_v=saved.lora_v, lora_vg=saved.lora_vg)

    def check_shapes(self, layer: MoeLayer, T: int):
        """Every buffer against the sizes a call with T tokens uses."""
        _routing_shapes(layer, T, self)
        R = T * layer.k
        _shape(self.checkpoint.codes, (R, 2 * layer.I), torch.uint8, "checkpoint.codes")
        _shape(self.checkpoint.scales, (R, layer.I // 16), torch.uint8, "checkpoint.scales")
        _shape(self.lora_v, (R, layer.lora_rank), torch.float32, "lora_v", optional=layer.lora_A is None)
        _shape(self.lora_vg, (R, layer.lora_rank), torch.float32, "lora_vg", optional=layer.lora_gu_A is None)

    def restore(self) -> SavedState:
        """The bf16 state that a backward reads."""
        h, a = swiglu_mxfp8_restore(self.checkpoint)
        return SavedState(**_fields(self), h=h, a=a, lora_v=self.lora_v, lora_vg=self.lora_vg)
