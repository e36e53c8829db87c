"""The plans of fp4_several.py, and the plan's model against the library's
workspaces."""
import pytest

import fp4_parts
from fp4_plan import STAGES, plan
from fp4_several import DIRECT, FORWARD, GRADIENT
from mxfp4_weight_mixture_02_amd import ops


def _up(v, a):
    return -(-v // a) * a


def _part_bytes(p):
    return _up(p.rest * p.splits * p.bn * p.bm * 4, 256)


@pytest.mark.parametrize("case", fp4_parts.FORWARD)
def test_the_model_gives_the_products_in_parts(case):
    p = plan(*case[:4], True)
    assert (p.bn, p.bm, p.rest, p.splits) == case[4:]


@pytest.mark.parametrize("case", fp4_parts.GRADIENT)
def test_the_model_gives_the_gradients_in_parts(case):
    M, N, K, f32 = case[:4]
    p = plan(M, N, _up(K, 64), f32, False)
    assert (p.bn, p.bm, p.rest, p.splits) == case[4:]


@pytest.mark.parametrize("case", FORWARD)
def test_products_take_several_tiles(case):
    M, N, K, f32 = case[:4]
    p = plan(M, N, K, f32, True)
    assert p.several and (p.tile, p.whole, p.rest, p.splits) == case[4:]
    assert -(-K // 256) > STAGES[0][p.tile]
    assert ops.lib().mxmoe_fp4_matmul_workspace_bytes(M, N, K, 0 if f32 else 1) == _part_bytes(p) + 256


@pytest.mark.parametrize("case", GRADIENT)
def test_gradients_take_several_tiles(case):
    M, N, K, f32 = case[:4]
    pad = _up(K, 64)
    p = plan(M, N, pad, f32, False)
    assert p.several and (p.tile, p.whole, p.rest, p.splits) == case[4:]
    assert pad // 64 > STAGES[1][p.tile]
    want = _up(N * pad * 2, 256) + _up(M * pad * 2, 256) + _part_bytes(p)
    assert ops.lib().mxmoe_fp4_linear_dx_workspace_bytes(M, K, N, 0 if f32 else 1) == want


def test_every_tile_that_may_have_several_does():
    # 128 x 128 and larger
    for cases, fp4 in ((FORWARD, True), (GRADIENT, False)):
        assert {(c[4], c[3]) for c in cases} == {(t, f) for t in range(5) for f in (False, True)}
        assert {c[4] for c in cases if c[6]} == set(range(5))


@pytest.mark.parametrize("M,N,K,f32,parts", DIRECT)
def test_gradients_straight_from_the_codes(M, N, K, f32, parts):
    want = (_up(parts * M * N * 4, 256) if parts > 1 else 0) + 256
    assert ops.lib().mxmoe_fp4_linear_dx_workspace_bytes(M, K, N, 0 if f32 else 1) == want
