"""Routing without a GPU: refusals of the C entry points and the binding,
and the float64 definition against closed forms and differences."""
import ctypes

import numpy as np
import pytest
import torch

import route_ref as ref
from mxfp4_weight_mixture_02_amd import Mxfp4Error, RouteOptions, moe_route, moe_route_backward, ops

FAKE = 0x10000   # never dereferenced: every call below returns from host checks
O = ops._RouteOpts


def _opts(**kw):
    d = dict(score=0, groups=1, top_groups=1, group_score=0, renorm=1, scale=1.0)
    d.update(kw)
    return O(**d)


def _route(o, T=4, E=16, k=2, logits=FAKE, idx=FAKE, ws=FAKE, n=1 << 20):
    return ops.lib().mxmoe_route(o, T, E, k, logits, None, idx, FAKE, FAKE, FAKE, ws, n, None)


@pytest.mark.parametrize("kw,call,code", [
    (dict(score=2), {}, -1), (dict(group_score=3), {}, -1), (dict(groups=0), {}, -1),
    (dict(groups=4, top_groups=5), {}, -1), (dict(top_groups=0), {}, -1),
    (dict(groups=3), {}, -2), (dict(groups=128, top_groups=128), dict(E=256), -2),
    (dict(groups=8, top_groups=1), dict(k=3), -2), (dict(scale=float("inf")), {}, -1),
    ({}, dict(T=0), -1), ({}, dict(k=0), -1), ({}, dict(E=0), -1), ({}, dict(E=300), -2),
    ({}, dict(E=4, k=5), -2), ({}, dict(k=9), -2), ({}, dict(T=1 << 26, k=4), -2),
    ({}, dict(T=1 << 62, k=4), -2),
    ({}, dict(logits=None), -1), ({}, dict(idx=None), -1), ({}, dict(logits=FAKE + 2), -1),
    ({}, dict(ws=None), -3), ({}, dict(n=16), -3), ({}, dict(ws=FAKE + 16), -1),
])
def test_route_refuses(kw, call, code):
    assert _route(_opts(**kw), **call) == code
    assert ops.lib().mxfp4_last_error()


def test_route_refuses_null_options():
    assert _route(None) == -1
    assert ops.lib().mxmoe_route_backward(None, 4, 16, 2, FAKE, FAKE, FAKE, FAKE, None) == -1
    assert ops.lib().mxmoe_route_backward(_opts(), 4, 16, 2, FAKE, None, FAKE, FAKE, None) == -1


@pytest.mark.parametrize("sizes", [(0, 16, 2), (4, 0, 1), (4, 300, 2), (4, 4, 5)])
def test_workspace_query_refuses(sizes):
    assert ops.lib().mxmoe_route_workspace_bytes(*sizes) == 0


def test_binding_refuses_shapes_and_devices():
    x = torch.zeros(4, 16)
    for match, call in [
            ("logits", lambda: moe_route(torch.zeros(16), 2)),
            ("logits", lambda: moe_route(x.double(), 2)),
            ("bias", lambda: moe_route(x, 2, bias=torch.zeros(15))),
            ("topk_idx", lambda: moe_route_backward(x, torch.zeros(4, 2), torch.zeros(4, 2))),
            ("topk_idx", lambda: moe_route_backward(x, torch.zeros(4, dtype=torch.int32), torch.zeros(4, 2))),
            ("dw", lambda: moe_route_backward(x, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 3))),
            ("CUDA tensor", lambda: moe_route(x, 2))]:
        with pytest.raises(ValueError, match=match):
            call()
    with pytest.raises(ValueError, match="score"):
        RouteOptions(score="relu")
    with pytest.raises(ValueError, match="group_score"):
        RouteOptions(group_score="mean")


def test_definition_by_hand():
    """Two groups; the better group by its two best, not by its best."""
    x = np.log(np.array([[1.0, 8.0, 5.0, 6.0]]))          # softmax: 0.05 0.4 0.25 0.3
    o = RouteOptions(groups=2, top_groups=1, group_score="top2", renorm=False)
    idx, w, off, rows = ref.route(x, 2, o)
    assert idx.tolist() == [[3, 2]] and np.allclose(w, [[0.3, 0.25]])
    idx, w, _, _ = ref.route(x, 2, RouteOptions(groups=2, top_groups=1))
    assert idx.tolist() == [[1, 0]] and np.allclose(w, [[8 / 9, 1 / 9]])
    assert off.tolist() == [0, 0, 0, 1, 2] and rows.tolist() == [1, 0]
    # the bias moves the choice and not the weight; equal values go by index
    o = RouteOptions(score="sigmoid", renorm=False, scale=2.0)
    idx, w, _, _ = ref.route(np.zeros((1, 3)), 2, o, bias=np.array([0.0, 0.0, 1.0], np.float32))
    assert idx.tolist() == [[2, 0]] and np.allclose(w, 1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_formula_against_differences(score, renorm):
    r = np.random.default_rng(3)
    o = RouteOptions(score=score, renorm=renorm, scale=1.5)
    x, idx, dw = r.normal(size=(1, 7)), np.array([[4, 0, 6]]), r.normal(size=(1, 3))
    g = ref.dlogits(x, idx, dw, o)[0]
    h = 1e-5
    for e in range(7):
        d = np.zeros(7)
        d[e] = h
        num = (ref.weights(x[0] + d, idx[0], o) - ref.weights(x[0] - d, idx[0], o)) @ dw[0] / (2 * h)
        # central differences: h^2 / 6 of a third derivative below 10, and 1e-16 / h of rounding
        assert abs(num - g[e]) < 1e-9


def test_router_logits_refuse():
    f = ops.lib().mxmoe_router_logits
    for args, code in [((0, 64, 8, FAKE, FAKE, None, FAKE), -1), ((4, 60, 8, FAKE, FAKE, None, FAKE), -2),
                       ((4, 64, 300, FAKE, FAKE, None, FAKE), -2), ((1 << 30, 64, 8, FAKE, FAKE, None, FAKE), -2),
                       ((1 << 25, 32, 256, FAKE, FAKE, None, FAKE), -2),
                       ((4, 64, 8, None, FAKE, None, FAKE), -1), ((4, 64, 8, FAKE + 8, FAKE, None, FAKE), -1)]:
        assert f(*args, None) == code and ops.lib().mxfp4_last_error()


def test_routed_block_refuses():
    from mxfp4_weight_mixture_02_amd.native import Dims, Grads, Saved, Weights
    d = Dims(T=16, H=64, I=64, E=4, k=2, swiglu_alpha=1.702, swiglu_limit=7.0)
    w = Weights(None, None, FAKE, FAKE, None, FAKE, FAKE, None)
    f, b = ops.lib().mxmoe_forward_routed, ops.lib().mxmoe_backward_routed
    routing = Saved(FAKE, FAKE, FAKE, FAKE)
    big = 1 << 40
    assert f(d, w, FAKE, FAKE, None, FAKE, big, None) == -1
    assert f(d, w, FAKE, FAKE, Saved(FAKE, FAKE, None, FAKE), FAKE, big, None) == -1
    assert f(d, w, FAKE, FAKE, Saved(FAKE, FAKE, FAKE, FAKE, FAKE), FAKE, big, None) == -1   # h without a
    assert f(d, w, FAKE, FAKE, routing, None, 0, None) == -3
    assert f(d, w, FAKE, None, routing, FAKE, big, None) == -1
    full = Saved(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE)
    g = Grads(dx=FAKE)
    assert b(d, w, full, None, FAKE, None, FAKE, FAKE, big, None) == -1
    assert b(d, w, full, None, FAKE, g, None, FAKE, big, None) == -1
    assert b(d, w, routing, None, FAKE, g, FAKE, FAKE, big, None) == -1
    assert b(d, w, full, None, FAKE, g, FAKE, None, 0, None) == -3
    assert b(d, w, full, None, FAKE, Grads(dx=FAKE, dW_gu=FAKE), FAKE, FAKE, big, None) == -1   # needs x


def test_routed_binding_refuses():
    import test_binding_host as th
    from mxfp4_weight_mixture_02_amd import (Routing, SavedState8, SwigluCheckpoint, mxfp4_moe_backward_routed,
                                             mxfp4_moe_forward, mxfp4_moe_forward_routed)
    layer, x, st = th._layer(), th._x(), th._saved(5)
    r = Routing(st.topk_idx, st.topk_w, st.expert_offsets, st.sorted_rows)
    eight = SavedState8(st.topk_idx, st.topk_w, st.expert_offsets, st.sorted_rows,
                        SwigluCheckpoint(torch.zeros(10, 192, dtype=torch.uint8), torch.zeros(10, 6, dtype=torch.uint8)))
    short = Routing(st.topk_idx, st.topk_w, st.expert_offsets[:-1], st.sorted_rows)
    for match, call in [("CUDA tensor", lambda: mxfp4_moe_forward_routed(layer, x, r)),
                        ("CUDA tensor", lambda: mxfp4_moe_forward_routed(th._layer(router_w=None), x, r)),
                        ("expert_offsets", lambda: mxfp4_moe_forward_routed(layer, x, short)),
                        ("topk_idx", lambda: mxfp4_moe_forward_routed(layer, th._x(6), r)),
                        ("mxfp8", lambda: mxfp4_moe_forward_routed(layer, x, r, saved="int8")),
                        ("mxfp8", lambda: mxfp4_moe_forward_routed(layer, x, r, saved=st)),
                        ("mxfp8", lambda: mxfp4_moe_forward(layer, x, saved="int8")),
                        ("a forward writes a SavedState", lambda: mxfp4_moe_forward(layer, x, saved=eight)),
                        ("router_w", lambda: mxfp4_moe_forward(th._layer(router_w=None), x)),
                        ("x is required", lambda: mxfp4_moe_backward_routed(layer, st, x, base=True)),
                        ("CUDA tensor", lambda: mxfp4_moe_backward_routed(layer, st, x))]:
        with pytest.raises(ValueError, match=match):
            call()
