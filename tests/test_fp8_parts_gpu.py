"""8-bit products in parts of K, in every tile: equal to products in 64 bits.

Elements are integers up to 3 times 1/2, 1 or 2 for each block, so a sum of
33885 products is below 33885 * 36, in steps of 1/4: less than 2^23 steps, which
an fp32 sum holds in any order.  In bf16 a K block's products of a row and a
column share a scale and are integers up to 9 times it, of which the scaled
matrix core drops nothing."""
import pytest
import torch

from fp8_parts import PARTS
from mxfp4_weight_mixture_02_amd import fp8_matmul, fp8_quantize

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("case", PARTS)
def test_parts_are_exact(case):
    M, N, K, f32 = case[:4]
    print("parts", case, flush=True)
    g = torch.Generator(device=DEV).manual_seed(M + 3 * N + 7 * K)

    def draw(rows, per):
        v = torch.randint(-3, 4, (rows, K), generator=g, device=DEV).float()
        e = torch.randint(-1, 2, (-(-rows // per), -(-K // 128)), generator=g, device=DEV).float().exp2()
        return v * e.repeat_interleave(per, 0)[:rows].repeat_interleave(128, 1)[:, :K]

    x = draw(M, 1)
    q, bias = fp8_quantize(x), torch.randint(-8, 9, (N,), generator=g, device=DEV).bfloat16()
    for rows in (128, 1):
        w = draw(N, rows)
        W = fp8_quantize(w, rows)
        want = (x.double() @ w.double().t() + bias.double()).float()
        del w
        y = fp8_matmul(q, W, bias=bias, dtype=torch.float32 if f32 else torch.bfloat16)
        assert torch.equal(y, want if f32 else want.bfloat16())
        assert torch.equal(y, fp8_matmul(q, W, bias=bias, dtype=y.dtype))
