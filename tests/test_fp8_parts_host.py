"""The sizes of fp8_parts.py are computed as it says: a product's workspace is
its fp32 parts, rounded up to 256 bytes, and 256 bytes more."""
import pytest

from fp8_parts import PARTS
from mxfp4_weight_mixture_02_amd import ops


@pytest.mark.parametrize("case", PARTS)
def test_workspace_holds_the_parts(case):
    M, N, K, f32, bn, bm, tiles, parts = case
    want = -(-tiles * parts * bn * bm * 4 // 256) * 256 + 256
    assert ops.lib().mxmoe_fp8_matmul_workspace_bytes(M, N, K, 0 if f32 else 1) == want
    whole = -(-M // bm) * -(-N // bn) - tiles
    assert whole >= 0
