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
from .native import Mxfp4Error, _shape

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
        for n in ("route", "route_backward"):
            getattr(L, "mxmoe_" + n).restype = ctypes.c_int
        _lib = L
    return _lib


def _same_device(**tensors):
    """Every tensor contiguous and on one GPU; returns that device."""
    dev = None
    for name, t in tensors.items():
        if t is None:
            continue
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"{name} is on {t.device}, other tensors on {dev}")
    return dev


def _call(name, dev, *args):
    """lib().<name>(*args, stream) on dev and its current stream."""
    fn = getattr(lib(), name)
    if torch.cuda.current_device() == dev.index:
        rc = fn(*args, torch._C._cuda_getCurrentRawStream(dev.index))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, torch._C._cuda_getCurrentRawStream(dev.index))
    if rc != native.MXFP4_OK:
        raise Mxfp4Error(name, rc, lib().mxfp4_last_error().decode())


def _p(t):
    return None if t is None else t.data_ptr()


def _bytes_needed(name, *args):
    n = getattr(lib(), name)(*args)
    if n == 0:
        raise Mxfp4Error(name, -1, lib().mxfp4_last_error().decode())
    return n


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
    nbytes = _bytes_needed("mxmoe_route_workspace_bytes", T, E, k)
    i32 = dict(dtype=torch.int32, device=dev)
    r = Routing(torch.empty((T, k), **i32), torch.empty((T, k), dtype=torch.float32, device=dev),
                torch.empty(E + 1, **i32), torch.empty(T * k, **i32))
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
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
