"""4-bit products and input gradients whose workgroups take several tiles, whose
copies run on from one tile into the next: equal to products in 64 bits.

Elements are integers up to 3 times 1/2, 1 or 2 for each block of 32, or (of dy)
integers up to 6: a sum of 12000 products is below 12000 * 36 in steps of 1/4,
less than 2^21 steps, which an fp32 sum holds in any order."""
import pytest
import torch

import fp4_ref as ref
from fp4_several import DIRECT, FORWARD, GRADIENT
from mxfp4_weight_mixture_02_amd import fp4_linear_dx, fp4_matmul, fp4_quantize

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF = torch.float32, torch.bfloat16


def _gen(case):
    return torch.Generator(device=DEV).manual_seed(case[0] + 3 * case[1] + 7 * case[2])


def _equal(got, left, right, bias, dtype):
    """got is left @ right + bias, its rows some at a time."""
    right = right.double()
    for a in range(0, got.shape[0], 8192):
        want = left[a:a + 8192].double() @ right
        if bias is not None:
            want += bias.double()
        assert torch.equal(got[a:a + 8192], want.float().to(dtype)), a


@pytest.mark.parametrize("case", FORWARD)
def test_products_are_exact(case):
    print("several", case, flush=True)
    M, N, K, f32 = case[:4]
    g = _gen(case)
    x, w = ref.whole(M, K, g, DEV, 1), ref.whole(N, K, g, DEV, 1)
    bias = torch.randint(-8, 9, (N,), generator=g, device=DEV).bfloat16()
    dtype = F32 if f32 else BF
    X, W = fp4_quantize(x), fp4_quantize(w)
    y = fp4_matmul(X, W, bias=bias, dtype=dtype)
    _equal(y, x, w.t(), bias, dtype)
    assert torch.equal(y, fp4_matmul(X, W, bias=bias, dtype=dtype))


@pytest.mark.parametrize("case", GRADIENT + DIRECT)
def test_gradients_are_exact(case):
    print("several", case, flush=True)
    M, N, K, f32 = case[:4]
    g = _gen(case)
    w = ref.whole(K, N, g, DEV, 1)
    dy = torch.randint(-6, 7, (M, K), generator=g, device=DEV).bfloat16()
    dtype = F32 if f32 else BF
    W = fp4_quantize(w)
    dx = fp4_linear_dx(dy, W, dtype=dtype)
    _equal(dx, dy, w, None, dtype)
    assert torch.equal(dx, fp4_linear_dx(dy, W, dtype=dtype))
