"""4-bit products and input gradients in parts of K, in every tile: equal to
products in 64 bits.

Elements are integers up to 3 times 1/2, 1 or 2 for each block of 32, or (of dy)
integers up to 6: a sum of 35000 products is below 35000 * 36 in steps of 1/4,
less than 2^23 steps, which an fp32 sum holds in any order."""
import pytest
import torch

import fp4_ref as ref
from fp4_parts import FORWARD, GRADIENT
from mxfp4_weight_mixture_02_amd import fp4_linear_dx, fp4_matmul, fp4_quantize

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF = torch.float32, torch.bfloat16


def _gen(case):
    return torch.Generator(device=DEV).manual_seed(case[0] + 3 * case[1] + 7 * case[2])


@pytest.mark.parametrize("case", FORWARD)
def test_products_in_parts_are_exact(case):
    print("parts", case, flush=True)
    M, N, K, f32 = case[:4]
    g = _gen(case)
    x, w = ref.whole(M, K, g, DEV, 1), ref.whole(N, K, g, DEV, 1)
    bias = torch.randint(-8, 9, (N,), generator=g, device=DEV).bfloat16()
    dtype = F32 if f32 else BF
    want = (x.double() @ w.double().t() + bias.double()).float().to(dtype)
    X, W = fp4_quantize(x), fp4_quantize(w)
    y = fp4_matmul(X, W, bias=bias, dtype=dtype)
    assert torch.equal(y, want) and torch.equal(y, fp4_matmul(X, W, bias=bias, dtype=dtype))


@pytest.mark.parametrize("case", GRADIENT)
def test_gradients_in_parts_are_exact(case):
    print("parts", case, flush=True)
    M, N, K, f32 = case[:4]
    g = _gen(case)
    w = ref.whole(K, N, g, DEV, 1)
    dy = torch.randint(-6, 7, (M, K), generator=g, device=DEV).bfloat16()
    dtype = F32 if f32 else BF
    want = (dy.double() @ w.double()).float().to(dtype)
    W = fp4_quantize(w)
    dx = fp4_linear_dx(dy, W, dtype=dtype)
    assert torch.equal(dx, want) and torch.equal(dx, fp4_linear_dx(dy, W, dtype=dtype))
