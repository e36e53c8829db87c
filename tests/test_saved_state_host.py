"""A saved state is what has the methods of one: a program's own class in the
place of SavedState is taken by every entry point that takes that."""
import pytest
import torch

import test_binding_host as th
from mxfp4_weight_mixture_02_amd import (SavedState8, SwigluCheckpoint, mxfp4_moe_backward, mxfp4_moe_backward_dx,
                                         mxfp4_moe_backward_routed, mxfp4_moe_forward, mxfp4_moe_forward_noalloc)


class Own:
    """Buffers of another state, kept by the program."""

    def __init__(self, state):
        self._state = state

    def check_shapes(self, layer, T):
        self._state.check_shapes(layer, T)

    def struct(self):
        return self._state.struct()

    def __getattr__(self, name):
        if name == "restore":
            raise AttributeError(name)
        return getattr(self._state, name)


def test_own_state_is_taken():
    layer, x, st = th._layer(), th._x(), Own(th._saved(5))
    for call in (lambda: mxfp4_moe_forward(layer, x, saved=st),
                 lambda: mxfp4_moe_forward_noalloc(layer, x, torch.empty_like(x), saved=st),
                 lambda: mxfp4_moe_backward_dx(layer, st, x),
                 lambda: mxfp4_moe_backward(layer, st, x, x),
                 lambda: mxfp4_moe_backward_routed(layer, st, x)):
        with pytest.raises(ValueError, match="CUDA tensor"):   # past every check of the state
            call()


def test_states_that_a_forward_cannot_write():
    layer, x, st = th._layer(), th._x(), th._saved(5)
    eight = SavedState8(st.topk_idx, st.topk_w, st.expert_offsets, st.sorted_rows,
                        SwigluCheckpoint(torch.zeros(10, 192, dtype=torch.uint8), torch.zeros(10, 6, dtype=torch.uint8)))
    for bad in (eight, {"h": st.h}):
        for call in (lambda: mxfp4_moe_forward(layer, x, saved=bad),
                     lambda: mxfp4_moe_forward_noalloc(layer, x, torch.empty_like(x), saved=bad)):
            with pytest.raises(ValueError, match="a forward writes a SavedState"):
                call()
    with pytest.raises(ValueError, match="expert_offsets"):
        mxfp4_moe_forward(layer, x, saved=Own(th._saved(5, expert_offsets=st.expert_offsets[:-1])))


def test_a_layers_own_check():
    """A layer class whose check takes no argument, as before routed calls."""
    class Layer(th.MoeLayer):
        def check_shapes(self):
            super().check_shapes()

    base = th._layer()
    layer = Layer(**{n: getattr(base, n) for n in base.__dataclass_fields__})
    with pytest.raises(ValueError, match="CUDA tensor"):
        layer.weights()
    with pytest.raises(ValueError, match="router_w is required"):
        Layer(**{**{n: getattr(base, n) for n in base.__dataclass_fields__}, "router_w": None}).weights()
