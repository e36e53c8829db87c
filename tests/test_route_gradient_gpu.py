"""The routing's gradient in both of its layouts (one token a wave, and from
4096 tokens on with E % 4 == 0 four tokens a wave), all rows against float64.

A gradient is an fp64 value rounded once to fp32: 1e-7 relative, plus 1e-12 of
the largest term of a row's sums for cancellation (fp64 steps of 1e-16, and an
exponential good to 1e-15, over at most 8 terms)."""
import numpy as np
import pytest
import torch

import route_grad_ref as ref
from mxfp4_weight_mixture_02_amd import RouteOptions, moe_route_backward

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

OPTIONS = [RouteOptions(), RouteOptions(renorm=False, scale=2.5), RouteOptions(score="sigmoid", scale=2.5),
           RouteOptions(score="sigmoid", renorm=False)]
EDGES = 14


def _edges(x, idx, rows):
    """Rows of -inf, of one number among -inf, NaN, infinities, scores of 0,
    lowest values; an index repeated, indices outside the experts."""
    E = x.shape[1]
    for i, r in enumerate(rows):
        if i == 0:
            x[r] = -np.inf
        elif i == 1:
            x[r, 1:] = -np.inf
        elif i == 2:
            x[r, E // 2] = np.nan
        elif i == 3:
            x[r] = np.nan
        elif i == 4:
            x[r, idx[r, 0]] = np.inf
        elif i == 5:
            x[r] = -800.0
        elif i == 6:
            x[r] = np.finfo(np.float32).min
        elif i == 7:
            idx[r] = idx[r, 0]
        elif i == 8:
            idx[r, 0], idx[r, -1] = -1, E
        elif i == 9:
            idx[r] = np.iinfo(np.int32).min
        elif i == 10:
            idx[r] = np.iinfo(np.int32).max
        elif i == 11:
            x[r, idx[r]] = -np.inf
        elif i == 12:
            x[r, idx[r, -1]] = np.nan
        elif i == 13:
            idx[r, -1] = idx[r, 0]


def _backward(x, idx, dw, o):
    return moe_route_backward(*(torch.from_numpy(np.ascontiguousarray(v)).to(DEV) for v in (x, idx, dw)), o)


@pytest.mark.parametrize("T", [EDGES, 4096 + 3, 4096 + 2 * 16 + 5])
@pytest.mark.parametrize("E", [4, 48, 64, 66, 100, 128, 130, 200, 256])
@pytest.mark.parametrize("o", range(len(OPTIONS)))
def test_all_rows(T, E, o):
    """Edge rows at the start, in the last workgroup, and at the very end."""
    print("route gradient", T, E, o, flush=True)
    r, k, o = np.random.default_rng(T + 3 * E), min(8, E), OPTIONS[o]
    x, dw = (r.normal(size=(T, E)) * 2).astype(np.float32), r.normal(size=(T, k)).astype(np.float32)
    idx = np.argsort(r.random(size=(T, E)), axis=1)[:, :k].astype(np.int32)
    _edges(x, idx, range(EDGES))
    if T > 2 * EDGES:
        _edges(x, idx, range(T - EDGES, T))
    got, want = _backward(x, idx, dw, o).cpu().numpy(), ref.dlogits(x, idx, dw, o)
    assert np.isfinite(want).any() and np.isnan(want).any()
    np.testing.assert_allclose(got, want, rtol=1e-7, atol=1e-12 * np.abs(dw).max() * o.scale * k)


@pytest.mark.parametrize("T", [50, 4100])
@pytest.mark.parametrize("E", [32, 66, 128, 256])
@pytest.mark.parametrize("gap", [300, 700, 709, 715, 725, 735, 800])
def test_scores_below_the_normal_range(T, E, gap):
    """The chosen experts' scores are e^-gap, below 2^-1022 from 709 on: their
    renormalised weights are ordinary numbers, and so is the gradient.  From
    746 on the scores are 0, and so are weights and gradient."""
    print("route gradient, small scores", T, E, gap, flush=True)
    r, o = np.random.default_rng(gap + E), RouteOptions(scale=1.5)
    x = np.zeros((T, E), np.float32)
    x[:, :3] = r.normal(size=(T, 3)) - gap
    idx, dw = np.tile(np.int32([2, 0, 1]), (T, 1)), r.normal(size=(T, 3)).astype(np.float32)
    got = _backward(x, idx, dw, o).cpu().numpy().astype(np.float64)
    assert np.all(got[:, 3:] == 0)
    s = np.take_along_axis(ref.scores(x, "softmax"), idx, 1).sum(1)
    if gap == 800:
        assert np.all(s == 0) and np.all(got == 0)
        return
    # The rounding to fp32; and each score off by 2^-50 of it and by at most two
    # steps of 2^-1074, which moves a weight by at most four times that over
    # the sum, and p by scale (|dw| + |dot|) of a weight's shift and scale w
    # times the three shifts in dot: at most 5 scale max |dw| in all.
    err = 4 * (2.0 ** -50 + 2 * 2.0 ** -1074 / s)
    _, p = ref.chosen_softmax(x, idx, dw, o)
    tol = 2.0 ** -24 * np.abs(p) + (5 * err * o.scale * np.abs(dw).max(1))[:, None]
    assert np.all(np.abs(np.take_along_axis(got, idx, 1) - p) <= tol)
