"""Sizes at the end of a launch (2^32 threads) are refused before anything is
enqueued, and the largest that are allowed are not refused as sizes."""
import pytest

from mxfp4_weight_mixture_02_amd import ops

FAKE = 0x10000   # never dereferenced: the calls below return from host checks
BIG = 1 << 60
UNSUPPORTED = -2


@pytest.mark.parametrize("T,E", [((1 << 26) - 1, 16), ((1 << 26) - 15, 1), ((1 << 25) - 3, 32)])
def test_router_logits_refuse(T, E):
    """1024 threads for 16 x 16 logits."""
    assert ops.lib().mxmoe_router_logits(T, 32, E, FAKE, FAKE, None, FAKE, None) == UNSUPPORTED


@pytest.mark.parametrize("M", [1, 16])
@pytest.mark.parametrize("N", [(1 << 27) - 15, (1 << 27) - 1])
def test_products_of_few_rows_refuse(M, N):
    """512 threads for 16 rows of W."""
    L = ops.lib()
    for K in (128, 250):
        assert L.mxmoe_fp8_linear(M, N, K, FAKE, FAKE, FAKE, None, 1, FAKE, FAKE, BIG, None) == UNSUPPORTED
        assert L.mxmoe_fp8_matmul(M, N, K, FAKE, FAKE, FAKE, FAKE, 128, None, 1, FAKE, FAKE, BIG, None) == UNSUPPORTED
        assert L.mxmoe_fp8_linear_workspace_bytes(M, N, K, 1) == L.mxmoe_fp8_matmul_workspace_bytes(M, N, K, 1) == 0
    assert L.mxmoe_fp8_matmul_workspace_bytes(M, (1 << 27) - 16, 128, 1) > 0
    # the weights' gradient has its rows and columns the other way round
    assert L.mxmoe_fp8_linear_dw_workspace_bytes(64, M, N) == 0


@pytest.mark.parametrize("R,I", [((1 << 30) - 1, 16), ((1 << 29) - 1, 32), ((1 << 34) // 48 - 1, 48)])
def test_swiglu_refuses(R, I):
    """A thread for 8 elements, in whole workgroups of 256."""
    n = (R, I, 1.702, 7.0)
    L = ops.lib()
    assert L.mxmoe_swiglu8_forward(FAKE, *n, FAKE, FAKE, FAKE, None) == UNSUPPORTED
    assert L.mxmoe_swiglu8_backward(FAKE, FAKE, FAKE, *n, FAKE, FAKE, None) == UNSUPPORTED
    assert L.mxmoe_swiglu8_restore(FAKE, FAKE, *n, FAKE, FAKE, None) == UNSUPPORTED
