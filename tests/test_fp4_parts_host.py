"""The sizes of fp4_parts.py are computed as it says: a workspace holds the
fp32 parts and, of a gradient, the bf16 operands, each rounded up to 256 bytes."""
import pytest

from fp4_parts import FORWARD, GRADIENT
from mxfp4_weight_mixture_02_amd import ops


def _up(v, a):
    return -(-v // a) * a


@pytest.mark.parametrize("case", FORWARD)
def test_a_products_workspace_holds_the_parts(case):
    M, N, K, f32, bn, bm, tiles, parts = case
    want = _up(tiles * parts * bn * bm * 4, 256) + 256
    assert ops.lib().mxmoe_fp4_matmul_workspace_bytes(M, N, K, 0 if f32 else 1) == want
    assert -(-M // bm) * -(-N // bn) >= tiles


@pytest.mark.parametrize("case", GRADIENT)
def test_a_gradients_workspace_holds_the_parts(case):
    M, N, K, f32, bn, bm, tiles, parts = case
    pad = _up(K, 64)
    want = _up(N * pad * 2, 256) + _up(M * pad * 2, 256) + _up(tiles * parts * bn * bm * 4, 256)
    assert ops.lib().mxmoe_fp4_linear_dx_workspace_bytes(M, K, N, 0 if f32 else 1) == want
    assert -(-M // bm) * -(-N // bn) >= tiles
