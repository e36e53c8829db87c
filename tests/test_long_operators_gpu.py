"""Norms, balance losses and 4-bit products of tensors whose offsets pass 2^32
bytes or elements: rows are the bits of calls on slices of them, which begin at
an offset of 0, and sums are compared with torch's in 64 bits."""
import pytest
import torch

import fp4_ref as ref
from mxfp4_weight_mixture_02_amd import (Fp4Matrix, fp4_linear, fp4_linear_dx, fp4_matmul, fp4_quantize, moe_balance,
                                         moe_balance_backward, rms_norm, rms_norm_backward)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF = torch.float32, torch.bfloat16
ROWS, WIDE = 1048700, 4200   # 1.03 x 2^32 elements


@pytest.fixture(autouse=True)
def _memory():
    yield
    torch.cuda.empty_cache()


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def test_norm():
    g = gen(0)
    x = torch.empty(ROWS, WIDE, dtype=BF, device=DEV).normal_(generator=g)
    w = torch.rand(WIDE, generator=g, device=DEV) + 0.5
    n = rms_norm(x, w, residual=x, fp8=True)
    # rows are split over waves alike from 1024 of them on
    ends = ((0, 1024), (ROWS // 2, ROWS // 2 + 1027), (ROWS - 1300, ROWS))
    for a, b in ends:
        s = rms_norm(x[a:b].clone(), w, residual=x[a:b].clone(), fp8=True)
        assert torch.equal(n.sum[a:b], s.sum) and torch.equal(n.rstd[a:b], s.rstd) and torch.equal(n.y[a:b], s.y)
        assert torch.equal(n.y8.codes[a:b], s.y8.codes) and torch.equal(n.y8.scales[:, a:b], s.y8.scales[:, :b - a])
    dx, dw = rms_norm_backward(n.y, n.sum, n.rstd, w, dsum=x)
    for a, b in ends:
        d, _ = rms_norm_backward(n.y[a:b].clone(), n.sum[a:b].clone(), n.rstd[a:b].clone(), w, dsum=x[a:b].clone())
        assert torch.equal(dx[a:b], d)
    del dx
    want, size = torch.zeros(2, WIDE, dtype=torch.float64, device=DEV)
    for a in range(0, ROWS, 1 << 16):
        t = n.sum[a:a + (1 << 16)].double() * n.rstd[a:a + (1 << 16), None].double() * n.y[a:a + (1 << 16)].double()
        want += t.sum(0)
        size += t.abs().sum(0)
    # two fp32 roundings a term, sums of at most 1025 rows in each of 1024
    # workgroups, then of these parts
    assert torch.all((dw.double() - want).abs() <= (2 + 1025 + 1024) * 2.0 ** -24 * size)


def test_balance():
    T, E, k = (1 << 24) + 77, 256, 2
    g = gen(1)
    x = torch.empty(T, E, device=DEV).normal_(generator=g)
    idx = torch.randint(0, E, (T, k), generator=g, device=DEV, dtype=torch.int32)
    out = moe_balance(x, idx)
    assert torch.equal(out.counts[0].long(), torch.bincount(idx.flatten().long(), minlength=E))
    assert out.tokens.tolist() == [T]
    # sums of 1024 tokens in fp32, 42 additions deep (3e-6 with the terms' own
    # errors), the others in fp64
    prob, z = torch.zeros(E, dtype=torch.float64, device=DEV), 0.0
    for a in range(0, T, 1 << 20):
        v = x[a:a + (1 << 20)].double()
        prob += v.softmax(1).sum(0)
        z += float(v.logsumexp(1).square().sum())
    assert torch.all((out.prob[0].double() - prob / T).abs() <= 1e-5 * prob / T)
    assert abs(float(out.losses[1]) - z / T) <= 1e-5 * z / T
    dl = torch.tensor([1.0, 0.5], device=DEV)
    d = moe_balance_backward(x, out, dl)
    for a, b in ((0, 99), ((1 << 24) - 31, T)):
        assert torch.equal(d[a:b], moe_balance_backward(x[a:b].clone(), out, dl))   # with the batch's counts


def test_rows_of_a_product():
    M, N, K = ROWS, 40, 8400
    g = gen(2)
    x = torch.empty(M, K, dtype=BF, device=DEV).normal_(generator=g)
    W = fp4_quantize(torch.randn(N, K, generator=g, device=DEV))
    y, X = fp4_linear(x, W, dtype=F32), fp4_quantize(x)
    assert torch.equal(y, fp4_matmul(X, W, dtype=F32))
    # in any order of the sums
    for a, b in ((0, 64), (M - 130, M)):
        q = fp4_quantize(x[a:b].clone())
        assert torch.equal(X.codes[a:b], q.codes)
        u, v = (torch.from_numpy(ref.values(m)).to(DEV) for m in (q, W))
        assert torch.all((y[a:b].double() - u @ v.t()).abs() <= (u.abs() @ v.abs().t()) * K * 2.0 ** -23)


@pytest.mark.parametrize("M", [3, 40, 130])
def test_rows_of_weights(M):
    """And the weights' transpose, 17 GB in bf16, of the gradient."""
    N, K = ROWS, 8400
    g = gen(3)
    codes = torch.randint(0, 256, (N, 4224), generator=g, device=DEV, dtype=torch.uint8)
    codes[:, 4200:] = 0
    # scales of 1: weights of up to 6 in steps of 1/2
    scales = torch.full((33, 4, ROWS // 16 * 16 + 16, 2), 127, dtype=torch.uint8, device=DEV)
    scales[:, :, N:] = 0
    W = Fp4Matrix(codes, scales, K)
    x = torch.randint(-3, 4, (M, K), generator=g, device=DEV).bfloat16()
    value = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], device=DEV)

    def rows(a, b):
        c = codes[a:b, :4200].int()
        return torch.stack((value[c & 15], value[c >> 4]), 2).view(b - a, K)

    y = fp4_linear(x, W, dtype=F32)
    dy = torch.randint(-1, 2, (M, N), generator=g, device=DEV).bfloat16()
    dx = torch.zeros(M, K, dtype=torch.float64, device=DEV)
    for a in range(0, N, 1 << 16):
        b = min(a + (1 << 16), N)
        w = rows(a, b).double()
        assert torch.equal(y[:, a:b], (x.double() @ w.t()).float())   # below 2^24 steps of 1/2
        dx += dy[:, a:b].double() @ w
    # a million products up to 6 in steps of 1/2, of random signs: far below 2^24 steps
    assert dx.abs().max() < 2.0 ** 20
    assert torch.equal(fp4_linear_dx(dy, W, dtype=F32), dx.float())


def test_results():
    """70000 x 70000 in bf16."""
    M = N = 70000
    g = gen(4)
    x, w = ref.whole(M, 96, g, DEV), ref.whole(N, 96, g, DEV)
    y = fp4_linear(x.bfloat16(), fp4_quantize(w))
    for a in range(0, M, 10000):
        assert torch.equal(y[a:a + 10000], (x[a:a + 10000].double() @ w.double().t()).float().bfloat16())
    del y
    dy, w = torch.randint(-8, 9, (M, 96), generator=g, device=DEV).bfloat16(), ref.whole(96, N, g, DEV)
    dx = fp4_linear_dx(dy, fp4_quantize(w))
    for a in range(0, M, 10000):
        assert torch.equal(dx[a:a + 10000], (dy[a:a + 10000].double() @ w.double()).float().bfloat16())
