"""4-bit products on the GPU against float64.

Quantized bytes are equal.  Products of integers up to 3 times powers of two
are exact in fp32 in any order of the sums, so those are equal too; for
others an fp32 sum of K products is within K 2^-23 of the sum of their
magnitudes, and a bf16 result another 2^-8 of its value."""
import numpy as np
import pytest
import torch

import fp4_ref as ref
import fp8_ref
from mxfp4_weight_mixture_02_amd import (fp4_linear, fp4_linear_dx, fp4_matmul, fp4_matrix, fp4_quantize,
                                         mxfp4_dequantize, mxfp4_quantize, ops)
from oracle import mxfp4

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF = torch.float32, torch.bfloat16


def dev(x, dtype=F32):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(DEV).to(dtype)


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def gen(*seed):
    return torch.Generator(device=DEV).manual_seed(sum(v * 31 ** i for i, v in enumerate(seed)) % (1 << 31))


# ---------------------------------------------------------------- quantizer

SHAPES = [(1, 1), (1, 32), (3, 7), (16, 129), (17, 256), (130, 257), (300, 1000), (33, 2880)]


def _equal(q, x):
    codes, scales = ref.quantize(x)
    assert np.array_equal(ref.natural(q), scales)
    assert np.array_equal(q.codes.cpu().numpy(), codes)


@pytest.mark.parametrize("rows,K", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("shift", [0, 1])
def test_quantizer(rows, K, dtype, shift):
    print("quantize", rows, K, dtype, shift, flush=True)
    r = np.random.default_rng(rows + K)
    x = r.normal(size=(rows, K)) * np.exp2(r.integers(-20, 20, size=(rows, K)))
    x[r.random(size=x.shape) < 0.1] = 0
    x = fp8_ref.bf16(x)
    flat = torch.empty(rows * K + shift, dtype=dtype, device=DEV)
    t = flat[shift:].view(rows, K)
    t.copy_(dev(x))
    _equal(fp4_quantize(t), x)


def test_quantizer_edges():
    """Every midpoint (ties), the scale's borders, subnormals, the largest and
    the smallest values, -0, NaN and infinities, in both types."""
    mid = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], np.float32)
    x = np.zeros((48, 32), np.float32)
    x[0, :7], x[0, 7:14], x[0, 31] = mid, -mid, 6
    x[1, :7], x[1, 7:14], x[1, 31] = np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(9)), -6
    x[2] = x[0] * np.float32(2.0 ** 100)
    x[3] = x[0] * np.float32(2.0 ** -120)
    for i, v in enumerate([6, 6.001, 12, 0.75, 0.7501, 1.5, 1.5001, 3.0e38, 3.4028234e38, 1.1754944e-38, 1e-38, 1e-45,
                           3.0e-39, -0.0]):
        x[4 + i, :4] = [v, -v / 3, v / 13, v / 300]
    x[20, 5], x[21, 6], x[22, 7] = np.nan, np.inf, -np.inf
    x[23, :] = np.nan
    x[24, 0], x[24, 1] = np.inf, 3.0
    with np.errstate(over="ignore"):
        for t, v in ((dev(x), x), (dev(x, BF), fp8_ref.bf16(x))):
            v = np.where(np.isnan(x), x, v)
            _equal(fp4_quantize(t), v)
            two = np.concatenate((v, v[::-1]), 1)   # a row's blocks keep to themselves
            _equal(fp4_quantize(torch.cat((t, t.flip(0)), 1)), two)


def test_quantizer_is_the_blocks():
    """The bytes of mxfp4_quantize, and its scales in the products' order."""
    g = gen(1)
    w = torch.randn(77, 352, generator=g, device=DEV) * torch.randn(77, 352, generator=g, device=DEV).exp()
    codes, scales = mxfp4_quantize(w)
    q, m = fp4_quantize(w), fp4_matrix(codes, scales)
    assert torch.equal(q.codes[:, :176], codes) and not q.codes[:, 176:].any()
    assert m.codes is codes and torch.equal(m.scales, q.scales)
    assert np.array_equal(ref.values(m), host(mxfp4_dequantize(codes, scales)))


# ------------------------------------------------------------------ products

PRODUCTS = [(1, 1, 1), (1, 17, 130), (2, 64, 128), (5, 33, 1000), (16, 16, 256), (16, 100, 2880), (17, 130, 260),
            (31, 40, 64), (33, 257, 384), (64, 128, 129), (65, 127, 100), (128, 128, 32), (129, 255, 640),
            (300, 500, 1312), (1, 5760, 2880), (64, 2880, 640), (700, 96, 33), (1, 1030, 96), (16, 2049, 160),
            (9, 1100, 2880), (3, 1030, 49152), (3, 1030, 50000), (13, 1500, 4000),
            (65, 130, 2880), (128, 129, 4000), (200, 40, 5024), (130, 1000, 777),
            # every tile, with rows and columns past its edge
            (4099, 2881, 96), (2050, 4101, 100), (4097, 1001, 640), (4100, 1001, 99), (2050, 1001, 1312),
            (2049, 1001, 288), (130, 8201, 100), (1030, 1001, 416), (33, 1001, 2880), (20, 2881, 2880),
            (2050, 7250, 2880), (3000, 5500, 2881), (1030, 7250, 5000), (8191, 2180, 160)]


@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_products_are_exact(M, N, K):
    """Blocks' magnitudes differ by powers of two, so that a scale at the wrong
    row or block shows.  |x| and |w| are below 12 in steps of 1/4: a sum of
    50000 products (standard deviation below 16 each) stays below 2^24 steps of
    1/16.  Both pitches of W, from 4-bit and from bf16 rows, both results."""
    print("product", M, N, K, flush=True)
    g = gen(M, N, K)
    x, w = ref.whole(M, K, g, DEV), ref.whole(N, K, g, DEV)
    bias = torch.randint(-8, 9, (N,), generator=g, device=DEV).bfloat16()
    want = (x.double() @ w.double().t()).float()
    full = (want.double() + bias.double()).float()
    X, W = fp4_quantize(x), fp4_quantize(w)
    ws = [W]
    if K % 32 == 0:
        ws.append(fp4_matrix(*mxfp4_quantize(w)))
        assert torch.equal(ws[1].scales, W.scales)
    xb = x.bfloat16()
    for v in ws:
        assert torch.equal(fp4_matmul(X, v, dtype=F32), want)
        assert torch.equal(fp4_linear(xb, v, dtype=F32), want)
        assert torch.equal(fp4_matmul(X, v, bias=bias), full.bfloat16())
        assert torch.equal(fp4_linear(xb, v, bias=bias), full.bfloat16())


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 64, 32), (2, 33, 96), (16, 100, 260), (65, 129, 100), (130, 64, 257),
                                   (70, 1000, 640), (300, 777, 1312), (2049, 1001, 288), (2050, 2881, 1001),
                                   (4099, 320, 2881), (33, 5760, 2880), (5000, 130, 64), (1030, 100, 8200),
                                   # up to 128 rows: one part of n and several, units and columns past the edges
                                   (1, 5760, 2880), (3, 70, 33000), (128, 333, 4064), (127, 8191, 160), (17, 1001, 8200),
                                   (100, 40001, 96), (129, 333, 4064), (64, 31, 2883), (8, 257, 31), (113, 256, 129)])
def test_input_gradients_are_exact(M, N, K):
    """dy of integers up to 8: sums of 5760 products below 2^24 steps of 1/4."""
    print("dx", M, N, K, flush=True)
    g = gen(M, N, K)
    w = ref.whole(N, K, g, DEV)
    dy = torch.randint(-8, 9, (M, N), generator=g, device=DEV).bfloat16()
    want = (dy.double() @ w.double()).float()
    ws = [fp4_quantize(w)] + ([fp4_matrix(*mxfp4_quantize(w))] if K % 32 == 0 else [])
    flat = torch.empty(M * N + 1, dtype=BF, device=DEV)
    odd = flat[1:].view(M, N)
    odd.copy_(dy)
    for v in ws:
        assert torch.equal(fp4_linear_dx(dy, v, dtype=F32), want)
        assert torch.equal(fp4_linear_dx(odd, v), want.bfloat16())


@pytest.mark.parametrize("M,N,K", [(1, 300, 2880), (16, 1200, 2880), (100, 320, 4096), (700, 1024, 2880)])
def test_random_products(M, N, K):
    r = np.random.default_rng(M)
    # blocks over many binades
    x = fp8_ref.bf16(r.normal(size=(M, K)) * np.repeat(np.exp2(r.integers(-12, 12, size=(M, -(-K // 32)))), 32, 1)[:, :K])
    w = r.normal(size=(N, K)).astype(np.float32)
    W = fp4_quantize(dev(w))
    X = fp4_quantize(dev(x, BF))
    a, b = ref.values(X), ref.values(W)
    want, size = a @ b.T, np.abs(a) @ np.abs(b).T
    tol = size * K * 2.0 ** -23
    for f in (lambda d: fp4_matmul(X, W, dtype=d), lambda d: fp4_linear(dev(x, BF), W, dtype=d)):
        assert np.all(np.abs(host(f(F32)) - want) <= tol)
        assert np.all(np.abs(host(f(BF)) - want) <= tol + np.abs(want) * 2.0 ** -8)
    dy = fp8_ref.bf16(r.normal(size=(M, N)))
    want, size = dy.astype(np.float64) @ b, np.abs(dy).astype(np.float64) @ np.abs(b)
    got = fp4_linear_dx(dev(dy, BF), W, dtype=F32)
    assert np.all(np.abs(host(got) - want) <= size * N * 2.0 ** -23)


def test_far_scales_and_small_values():
    """Blocks 2^200 apart in one row; results from 2^-126 on."""
    x = np.zeros((20, 256), np.float32)
    x[:, :32], x[:, 64:96] = 3 * 2.0 ** 100, 2.0 ** -100
    w = np.zeros((40, 256), np.float32)
    w[:20, 0], w[20:, 70] = 2.0 ** -90, 2.0 ** 90
    got = host(fp4_matmul(fp4_quantize(dev(x)), fp4_quantize(dev(w)), dtype=F32))
    assert np.all(got[:, :20] == 3 * 2.0 ** 10) and np.all(got[:, 20:] == 2.0 ** -10)
    one = np.ones((3, 32), np.float32)
    for e in (-126, -100, 100, 126):
        got = host(fp4_matmul(fp4_quantize(dev(one * 2.0 ** (e // 2))), fp4_quantize(dev(one * 2.0 ** (e - e // 2 - 5))),
                              dtype=F32))
        assert np.all(got == 2.0 ** e) or e == 126 and np.all(got == 2.0 ** 126)


@pytest.mark.parametrize("M,N", [(3, 40), (3, 1100), (20, 40), (300, 200), (2100, 1100)])
def test_a_nan_block_stays_in_its_row(M, N):
    K = 352
    x, w = ref.whole(M, K, gen(M), DEV), ref.whole(N, K, gen(N), DEV)
    x[M - 1, 340], w[N - 2, 3], w[7, 351] = torch.inf, torch.nan, torch.nan
    bad = torch.zeros(M, N, dtype=torch.bool, device=DEV)
    bad[M - 1], bad[:, N - 2], bad[:, 7] = True, True, True
    want = x.nan_to_num(0, 0, 0).double() @ w.nan_to_num(0, 0, 0).double().t()
    scales = ref.quantize(w.cpu().numpy())[1][:, :11]
    # K / 2 bytes a row: the last chunks of a row are followed by the next one's
    flat = fp4_matrix(fp4_quantize(w).codes[:, :176].contiguous(), torch.from_numpy(np.ascontiguousarray(scales)).to(DEV))
    for v in (fp4_quantize(w), flat):
        for y in (fp4_matmul(fp4_quantize(x), v, dtype=F32), fp4_linear(x.bfloat16(), v, dtype=F32)):
            assert torch.equal(torch.isnan(y), bad) and torch.equal(y[~bad].double(), want[~bad])
    dx = fp4_linear_dx(torch.ones(M, N, dtype=BF, device=DEV), flat, dtype=F32)
    cols = torch.zeros(K, dtype=torch.bool, device=DEV)
    cols[:32], cols[320:] = True, True
    assert torch.equal(torch.isnan(dx), cols.expand(M, K))


@pytest.mark.parametrize("M,N,K", [(5, 333, 352), (40, 1000, 96), (300, 130, 640), (2100, 320, 1100), (2100, 321, 1100)])
def test_a_nan_gradient_stays_in_its_row(M, N, K):
    g = gen(M, N, K)
    w = ref.whole(N, K, g, DEV)
    dy = torch.randint(-8, 9, (M, N), generator=g, device=DEV).bfloat16()
    want = (dy.double() @ w.double()).float()
    dy[1, 0], dy[3, N - 1], dy[M - 1, N - 1] = torch.nan, torch.nan, torch.nan
    got = fp4_linear_dx(dy, fp4_quantize(w), dtype=F32)
    bad = torch.zeros(M, dtype=torch.bool, device=DEV)
    bad[[1, 3, M - 1]] = True
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], want[~bad])


@pytest.mark.parametrize("M", [1, 20, 40, 1100])
@pytest.mark.parametrize("N,K", [(1, 40), (257, 352), (1001, 96), (1030, 288)])
def test_scales_past_the_rows_are_not_used(M, N, K):
    g = gen(M, N)
    x, w = ref.whole(M, K, g, DEV), ref.whole(N, K, g, DEV)
    dy = torch.randint(-8, 9, (M, N), generator=g, device=DEV).bfloat16()
    X, W = fp4_quantize(x), fp4_quantize(w)
    X.scales[:, :, M:], W.scales[:, :, N:] = 255, 255
    assert torch.equal(fp4_matmul(X, W, dtype=F32), (x.double() @ w.double().t()).float())
    assert torch.equal(fp4_linear(x.bfloat16(), W, dtype=F32), (x.double() @ w.double().t()).float())
    assert torch.equal(fp4_linear_dx(dy, W, dtype=F32), (dy.double() @ w.double()).float())


@pytest.mark.parametrize("M,N,K", [(3, 1030, 96), (33, 257, 352), (300, 130, 2880), (2050, 1001, 288)])
def test_nothing_else_is_written(M, N, K):
    G = 4096
    g = gen(M, N)
    x, w, dy = (torch.randn(s, generator=g, device=DEV).bfloat16() for s in ((M, K), (N, K), (M, N)))
    W = fp4_matrix(*mxfp4_quantize(w.float()))
    L, s, p = ops.lib(), torch.cuda.current_stream().cuda_stream, lambda t: t.data_ptr()
    for name, rows, cols, a, want in (("linear", M, N, x, fp4_linear(x, W)), ("linear_dx", M, K, dy, fp4_linear_dx(dy, W))):
        flat = torch.full((rows * cols + 2 * G,), 7.0, dtype=BF, device=DEV)
        n = getattr(L, f"mxmoe_fp4_{name}_workspace_bytes")(M, N, K, 1)
        ws = torch.full((n + 512,), 9, dtype=torch.uint8, device=DEV)
        args = [M, N, K, p(a), p(W.codes), K // 2, p(W.scales)] + ([None] if name == "linear" else [])
        assert getattr(L, "mxmoe_fp4_" + name)(*args, 1, p(flat) + 2 * G, p(ws), n, s) == 0
        assert torch.equal(flat[G:-G].view(rows, cols), want)
        assert torch.all(flat[:G] == 7) and torch.all(flat[-G:] == 7) and torch.all(ws[n:] == 9)


def test_streams_and_graphs():
    """Two graphs of a layer's step on streams of their own, replayed in turn
    with eager calls between, give the eager bits."""
    g = gen(5)
    H, I, T = 320, 288, 130
    wg = fp4_matrix(*mxfp4_quantize(torch.randn(2 * I, H, generator=g, device=DEV)))
    wd = fp4_matrix(*mxfp4_quantize(torch.randn(H, I, generator=g, device=DEV)))
    xs = [torch.randn(T, H, generator=g, device=DEV).bfloat16() for _ in range(3)]

    def step(x):
        out = []
        for rows in (x, x[:3].contiguous()):
            h = fp4_linear(rows, wg)
            y = fp4_linear(h[:, :I].contiguous(), wd, dtype=F32)
            out += [h, y, fp4_linear_dx(y.bfloat16(), wd), fp4_linear_dx(h, wg), fp4_matmul(fp4_quantize(rows), wg)]
        return out

    want = [step(x) for x in xs]
    hold = [xs[0].clone(), xs[1].clone()]
    graphs, outs = [], []
    for h in hold:
        gr, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(gr, stream=side):
            outs.append(step(h))
        graphs.append(gr)
    for i in range(4):
        for h, j in zip(hold, (i % 3, (i + 1) % 3)):
            h.copy_(xs[j])
        step(xs[2])
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for o, j in zip(outs, (i % 3, (i + 1) % 3)):
            assert all(torch.equal(a, b) for a, b in zip(o, want[j]))
