"""The batched reference of the routing and its gradient against the other
reference, differences and closed forms."""
import numpy as np
import pytest

import route_grad_ref as grad
import route_ref as ref
from mxfp4_weight_mixture_02_amd import RouteOptions

OPTIONS = [RouteOptions(), RouteOptions(renorm=False, scale=2.5), RouteOptions(score="sigmoid", scale=2.5),
           RouteOptions(score="sigmoid", renorm=False)]


@pytest.mark.parametrize("o", OPTIONS)
def test_gradient_is_the_formulas(o):
    r = np.random.default_rng(0)
    x, dw = r.normal(size=(50, 12)) * 2, r.normal(size=(50, 4))
    idx = r.integers(0, 12, size=(50, 4))   # with repetitions
    # float64 on both sides, terms up to |dw| scale
    np.testing.assert_allclose(grad.dlogits(x, idx, dw, o), ref.dlogits(x, idx, dw, o), rtol=1e-12, atol=1e-13)


@pytest.mark.parametrize("o", OPTIONS)
def test_gradient_against_differences(o):
    r = np.random.default_rng(1)
    x, idx, dw = r.normal(size=(1, 7)), np.array([[4, 0, 6]]), r.normal(size=(1, 3))
    g, h = grad.dlogits(x, idx, dw, o)[0], 1e-5
    for e in range(7):
        d = np.zeros(7)
        d[e] = h
        num = (ref.weights(x[0] + d, idx[0], o) - ref.weights(x[0] - d, idx[0], o)) @ dw[0] / (2 * h)
        # central differences: h^2 / 6 of a third derivative below 10, and 1e-16 / h of rounding
        assert abs(num - g[e]) < 1e-9


@pytest.mark.parametrize("gap", [10, 300, 700, 708, 715, 725, 735])
def test_scores_below_the_normal_range_have_a_gradient(gap):
    """Chosen softmax scores of e^-gap: their weights are ordinary numbers."""
    r = np.random.default_rng(gap)
    x = np.zeros((20, 6))
    x[:, :3] = r.normal(size=(20, 3)) - gap
    idx, dw, o = np.tile([2, 0, 1], (20, 1)), r.normal(size=(20, 3)), RouteOptions(scale=1.5)
    w, p = grad.chosen_softmax(x, idx, dw, o)
    g = grad.dlogits(x, idx, dw, o)
    # a score is off by 2^-52 and by at most two steps of 2^-1074 of its own
    s = np.take_along_axis(grad.scores(x, "softmax"), idx, 1)
    err = 2.0 ** -50 + 8 * 2.0 ** -1074 / s.sum(1).min()
    assert np.isfinite(g).all() and np.all(g[:, 3:] == 0)
    assert np.abs(np.take_along_axis(g, idx, 1) - p).max() <= 4 * err * o.scale * np.abs(dw).max() * 3


@pytest.mark.parametrize("o", OPTIONS + [RouteOptions(groups=4, top_groups=2), RouteOptions(score="sigmoid", groups=2)])
def test_routing_is_the_definitions(o):
    r = np.random.default_rng(2)
    x, bias = (r.integers(-6, 7, size=(60, 24)) / 2).astype(np.float32), r.normal(size=24).astype(np.float32) * 0.1
    for b in (None, bias):
        for a, want in zip(grad.route(x, 5, o, b), ref.route(x, 5, o, b)):
            if a.dtype == np.float64:
                np.testing.assert_allclose(a, want, rtol=1e-14)
            else:
                assert np.array_equal(a, want)
