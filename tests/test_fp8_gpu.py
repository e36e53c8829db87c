"""8-bit products and checkpoints on the GPU against float64.

Quantized bytes are equal.  Products of small integers are exact in fp32 in
any order of the sums, so they are equal too; for others an fp32 sum of K
products is within K 2^-23 of the sum of their magnitudes (every addition
rounds or cuts at 2^-23 of a partial sum at most that large), and a bf16
result another 2^-8 of its value.  SwiGLU outputs: bf16 (2^-8) of an fp32
value whose hardware exponential and reciprocal are good to about 2^-21."""
import numpy as np
import pytest
import torch

import fp8_ref as ref
from mxfp4_weight_mixture_02_amd import (fp8_linear, fp8_linear_dw, fp8_linear_dx, fp8_matmul, fp8_quantize,
                                         fp8_quantize_t, fp8_transpose, swiglu_mxfp8, swiglu_mxfp8_backward,
                                         swiglu_mxfp8_restore)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def dev(x, dtype=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(DEV).to(dtype)


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def wide(r, shape):
    """Values over many binades, zeros among them."""
    x = r.normal(size=shape) * np.exp2(r.integers(-20, 20, size=shape))
    x[r.random(size=shape) < 0.1] = 0
    return ref.bf16(x)


# ---------------------------------------------------------------- quantizers

SHAPES = [(1, 1), (1, 128), (3, 7), (16, 129), (17, 200), (130, 256), (300, 1000), (129, 72)]


def _equal(q, x, block_rows):
    codes, e, nan = ref.quantize(x, block_rows, 128)
    got = q.codes.cpu().numpy()
    assert np.array_equal(got | (nan_mask(got)), codes | nan_mask(codes))   # the NaN code's sign is free
    s = ref.scale_bytes(e, block_rows, x.shape[0])
    n = s.shape[1] if block_rows == 128 else x.shape[0]
    assert np.array_equal(q.scales.cpu().numpy()[:, :n], s[:, :n])


def nan_mask(c):
    return np.where((c & 0x7F) == 0x7F, 0x80, 0).astype(np.uint8)


@pytest.mark.parametrize("rows,K", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantizers(rows, K, dtype):
    print("quantize", rows, K, dtype, flush=True)
    x = wide(np.random.default_rng(rows + K), (rows, K))
    t = dev(x, dtype)
    _equal(fp8_quantize(t), x, 1)
    _equal(fp8_quantize(t, 128), x, 128)
    _equal(fp8_quantize_t(t), x.T, 1)
    w = fp8_quantize(t, 128)
    _equal(fp8_transpose(w), x.T, 128)


def test_quantize_misaligned_rows():
    """A base that is not 16-byte aligned takes the elementwise loads."""
    x = wide(np.random.default_rng(5), (33 * 40 + 1,))
    for dtype in (torch.float32, torch.bfloat16):
        t = dev(x, dtype)[1:].view(33, 40)
        _equal(fp8_quantize(t), x[1:].reshape(33, 40), 1)
        _equal(fp8_quantize_t(t), x[1:].reshape(33, 40).T, 1)


def test_quantize_edges():
    """Every fp8 midpoint (ties), the scale's borders, subnormals, the largest
    and the smallest values, NaN and infinities."""
    grid = ref.e4m3_decode(np.arange(0x7F))
    mid = (grid[:-1] + grid[1:]) / 2
    x = np.zeros((40, 128), np.float32)
    x[0, :126], x[0, 127] = mid, 448
    x[1, :126], x[1, 127] = -np.nextafter(mid.astype(np.float32), np.float32(0)), 448
    for i, v in enumerate([448, 448.5, 449, 0.875, 0.8751, 1.75, 3.0e38, 3.4028234e38, 1.1754944e-38, 1e-38, 1e-45]):
        x[2 + i, :3] = [v, -v / 3, v / 300]
    x[20, 5], x[21, 6], x[22, 7] = np.nan, np.inf, -np.inf
    x[23, :] = np.nan
    x[24, 0], x[24, 1] = np.inf, 3.0
    x[25, 0] = -0.0
    _equal(fp8_quantize(dev(x)), x, 1)
    _equal(fp8_quantize_t(dev(x)), x.T, 1)
    _equal(fp8_quantize(dev(x), 128), x, 128)


# ------------------------------------------------------------------ products

PRODUCTS = [(1, 1, 1), (1, 17, 130), (2, 64, 128), (5, 33, 1000), (16, 16, 256), (16, 100, 2880), (17, 130, 260),
            (31, 40, 64), (33, 257, 384), (64, 128, 129), (65, 127, 100), (128, 128, 128), (129, 255, 640),
            (300, 500, 1300), (1, 5760, 2880), (64, 2880, 640), (700, 96, 33),
            # few tiles: K split into parts and joined
            (65, 130, 2880), (128, 129, 4000), (200, 40, 5000), (130, 1000, 777)]


def _integers(r, shape, top=3):
    return r.integers(-top, top + 1, size=shape).astype(np.float32)




@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_integer_products_are_exact(M, N, K):
    """Block magnitudes differ by powers of two, so that a scale applied to
    the wrong row or block shows; all sums stay below 2^24 of the finest step."""
    print("product", M, N, K, flush=True)
    r = np.random.default_rng(M * 31 + N * 7 + K)
    x, w = _integers(r, (M, K)), _integers(r, (N, K))
    kb = -(-K // 128)
    xs = np.exp2(r.integers(-2, 3, size=(M, kb)).astype(np.float32))
    ws = np.exp2(r.integers(-2, 3, size=(-(-N // 128), kb)).astype(np.float32))
    wr = np.exp2(r.integers(-2, 3, size=(N, kb)).astype(np.float32))
    x = x * np.repeat(xs, 128, 1)[:, :K]
    wb = w * np.repeat(np.repeat(ws, 128, 0)[:N], 128, 1)[:, :K]
    wv = w * np.repeat(wr, 128, 1)[:, :K]
    bias = _integers(r, (N,))
    want, rows = x.astype(np.float64) @ wb.T, x.astype(np.float64) @ wv.T
    xb, q, W, V = dev(x, torch.bfloat16), fp8_quantize(dev(x)), fp8_quantize(dev(wb), 128), fp8_quantize(dev(wv))
    b = dev(bias, torch.bfloat16)
    f32 = torch.float32
    assert np.array_equal(host(fp8_matmul(q, W, dtype=f32)), want)
    assert np.array_equal(host(fp8_matmul(q, V, dtype=f32)), rows)
    assert np.array_equal(host(fp8_linear(xb, W, dtype=f32)), want)
    assert np.array_equal(host(fp8_linear(xb, W, bias=b, dtype=f32)), want + bias)
    assert torch.equal(fp8_linear(xb, W, bias=b), dev(want + bias, torch.bfloat16))
    assert torch.equal(fp8_matmul(q, V, bias=b), dev(rows + bias, torch.bfloat16))



# every tile of the products, with rows and columns past its edge, whole; parts
# of K in the smaller tiles, and a product whose last round alone is in parts
# (fp8_parts.py has every tile that is taken in parts)
TILES = [(4099, 2881, 100), (2050, 4101, 100), (4097, 1001, 640), (4100, 1001, 99), (2050, 1001, 1300),
         (2049, 1001, 100), (130, 8201, 100), (1030, 1001, 100), (33, 1001, 2881), (20, 2881, 2881),
         (3, 1030, 384), (16, 2049, 140), (5, 1100, 2880), (8, 1100, 2880), (2050, 7250, 2881), (3000, 5500, 2881), (1030, 7250, 5000)]


@pytest.mark.parametrize("M,N,K", TILES)
def test_tiles_are_exact(M, N, K):
    """Integers times block magnitudes, as above, against products in 64 bits:
    |x| and |w| stay below 12 in steps of 1/4, a sum of 5000 products below
    2^24 steps of 1/16."""
    print("tiles", M, N, K, flush=True)
    g = torch.Generator(device=DEV).manual_seed(M + 3 * N + 7 * K)

    def draw(rows, per):
        v = torch.randint(-3, 4, (rows, K), generator=g, device=DEV).float()
        e = torch.randint(-2, 3, (-(-rows // per), -(-K // 128)), generator=g, device=DEV).float().exp2()
        return v * e.repeat_interleave(per, 0)[:rows].repeat_interleave(128, 1)[:, :K]

    x, wb, wv = draw(M, 1), draw(N, 128), draw(N, 1)
    q = fp8_quantize(x)
    for w, rows in ((wb, 128), (wv, 1)):
        W = fp8_quantize(w, rows)
        want = x.double() @ w.double().t()
        assert torch.equal(fp8_matmul(q, W, dtype=torch.float32).double(), want)
        if rows == 128:
            assert torch.equal(fp8_linear(x.bfloat16(), W, dtype=torch.float32).double(), want)
        # bf16: a K block's products of a row and a column share a scale and
        # are integers up to 9, of which the scaled matrix core drops nothing
        assert torch.equal(fp8_matmul(q, W), want.float().bfloat16())


@pytest.mark.parametrize("M,N,K", [(1, 40, 33), (130, 129, 257), (511, 200, 640), (2049, 320, 96), (64, 16, 16),
                                   (5000, 100, 70), (3000, 66, 65)])
def test_integer_weight_gradients_are_exact(M, N, K):
    print("dw", M, N, K, flush=True)
    r = np.random.default_rng(M + N + K)
    mb = -(-M // 128)
    dy = _integers(r, (M, N)) * np.repeat(np.exp2(r.integers(-2, 3, size=(mb, N))), 128, 0)[:M]
    x = _integers(r, (M, K)) * np.repeat(np.exp2(r.integers(-2, 3, size=(mb, K))), 128, 0)[:M]
    got = fp8_linear_dw(dev(dy, torch.bfloat16), dev(x, torch.bfloat16))
    assert np.array_equal(host(got), dy.T.astype(np.float64) @ x)


def test_large_tiles_are_exact():
    """Sizes that take the largest tiles, ragged in all three."""
    g = torch.Generator(device=DEV).manual_seed(1)
    for M, N, K in [(4100, 4099, 300), (8191, 2180, 130)]:
        print("large", M, N, K, flush=True)
        x = torch.randint(-3, 4, (M, K), generator=g, device=DEV).to(torch.bfloat16)
        w = torch.randint(-3, 4, (N, K), generator=g, device=DEV).float()
        want = (x.double() @ w.double().t()).float()
        W = fp8_quantize(w, 128)
        assert torch.equal(fp8_linear(x, W, dtype=torch.float32), want)
        assert torch.equal(fp8_linear(x, W), want.bfloat16())
        assert torch.equal(fp8_matmul(fp8_quantize(x), fp8_quantize(w), dtype=torch.float32), want)
        dy = torch.randint(-3, 4, (K, N), generator=g, device=DEV).to(torch.bfloat16)
        xx = torch.randint(-3, 4, (K, M), generator=g, device=DEV).to(torch.bfloat16)
        assert torch.equal(fp8_linear_dw(dy, xx), (dy.double().t() @ xx.double()).float())


@pytest.mark.parametrize("M,N,K", [(1, 96, 2880), (16, 320, 520), (48, 130, 700), (200, 300, 1111)])
def test_products_forward_and_backward(M, N, K):
    """Ordinary values: fp8_linear, its input gradient with the transposed
    weights and its weight gradient, against float64 products of the rounded
    operands; and those against the unrounded formula within E4M3's 2^-4."""
    print("linear", M, N, K, flush=True)
    r = np.random.default_rng(N + K)
    x, dy = ref.bf16(r.normal(size=(M, K))), ref.bf16(r.normal(size=(M, N)))
    w, bias = r.normal(size=(N, K)).astype(np.float32) * 0.02, ref.bf16(r.normal(size=N))
    W = fp8_quantize(dev(w), 128)
    xq, wq, dq = ref.rounded(x), ref.rounded(w, 128), ref.rounded(dy)
    cases = [
        (fp8_linear(dev(x, torch.bfloat16), W, bias=dev(bias, torch.bfloat16)), xq @ wq.T + bias,
         np.abs(xq) @ np.abs(wq).T + np.abs(bias), K + 1, 2.0 ** -8),
        (fp8_linear_dx(dev(dy, torch.bfloat16), fp8_transpose(W)), dq @ wq, np.abs(dq) @ np.abs(wq), N, 2.0 ** -8),
        (fp8_linear_dx(dev(dy, torch.bfloat16), fp8_transpose(W), dtype=torch.float32), dq @ wq,
         np.abs(dq) @ np.abs(wq), N, 0.0),
        (fp8_linear_dw(dev(dy, torch.bfloat16), dev(x, torch.bfloat16)), ref.rounded(dy.T) @ ref.rounded(x.T).T,
         np.abs(dy.T) @ np.abs(x) * 1.2, M, 0.0)]
    for got, want, size, n, half in cases:
        assert np.all(np.abs(host(got) - want) <= n * 2.0 ** -23 * size + half * np.abs(want) * 1.01)
    # every rounded operand is within 2^-4 of its value (2^-9 * 2^e below the
    # normal range: 2^-10 of the block's 448 * 2^e at most, here well below)
    full = np.abs(x) @ np.abs(w).T
    assert np.all(np.abs(xq @ wq.T - x.astype(np.float64) @ w.T) <= full * (2 * 2.0 ** -4 + 2.0 ** -8) + 1e-2)


def test_nan_stays_in_its_row_and_scale_padding_is_unused():
    r = np.random.default_rng(2)
    for M in (3, 40, 200):
        x, w = r.normal(size=(M, 256)).astype(np.float32), r.normal(size=(130, 256)).astype(np.float32)
        x[1, 7], x[2, 200] = np.nan, np.inf
        for blocks in (1, 128):
            q, W = fp8_quantize(dev(x)), fp8_quantize(dev(w), blocks)
            q.scales[:, M:] = 255
            if blocks == 1:
                W.scales[:, 130:] = 255
            y = fp8_matmul(q, W)
            bad = torch.zeros(M, dtype=torch.bool, device=DEV)
            bad[1:3] = True
            assert torch.all(y[bad].isnan()) and torch.all(y[~bad].isfinite())


@pytest.mark.parametrize("M,K", [(1, 128), (2, 256), (3, 2944), (16, 384), (11, 2048), (13, 2688)])
def test_one_launch_form_where_the_last_elements_are_small(M, K):
    """The form for few rows rounds X itself: a row whose last 8 elements are
    far below its block's largest still has the block's scale."""
    r = np.random.default_rng(M)
    x = r.integers(-7, 8, size=(M, K)).astype(np.float32) * 32
    x[:, -8:] = [1, -1, 0.5, 2, 0.25, -0.5, 1, 1]
    w = _integers(r, (40, K))
    for dtype in (torch.float32, torch.bfloat16):
        y = fp8_linear(dev(x, torch.bfloat16), fp8_quantize(dev(w), 128), dtype=dtype)
        q = fp8_matmul(fp8_quantize(dev(x)), fp8_quantize(dev(w), 128), dtype=dtype)
        assert np.array_equal(host(q), host(y))
    assert np.array_equal(host(fp8_linear(dev(x, torch.bfloat16), fp8_quantize(dev(w), 128), dtype=torch.float32)),
                          ref.rounded(x) @ w.T.astype(np.float64))


def test_zeros_and_tiny_values():
    z = torch.zeros(20, 300, dtype=torch.bfloat16, device=DEV)
    W = fp8_quantize(torch.zeros(40, 300, device=DEV), 128)
    assert torch.all(fp8_linear(z, W) == 0)
    assert torch.all(fp8_linear_dw(z, z) == 0)
    for M in (4, 20, 100):   # 2^-100 * 2^90: one exact, the other operand's scale near its end
        x = torch.full((M, 128), 2.0 ** -100, dtype=torch.bfloat16, device=DEV)
        W = fp8_quantize(torch.full((16, 128), 2.0 ** 90, device=DEV), 128)
        assert torch.all(fp8_linear(x, W, dtype=torch.float32) == 2.0 ** -3)


def test_offsets_past_32_bits():
    """2.2e9 bytes of codes, and 2.2e9 outputs: the last rows are those of a
    small call, to two bf16 roundings (other sizes may sum in another order)."""
    def near(a, b):
        return torch.all((a.float() - b.float()).abs() <= 2.0 ** -7 * b.float().abs() + 1e-3)

    g = torch.Generator(device=DEV).manual_seed(0)
    x = torch.empty(540000, 4096, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    W = fp8_quantize(torch.empty(40, 4096, device=DEV).normal_(generator=g), 128)
    y = fp8_linear(x, W)
    assert near(y[-1000:], fp8_linear(x[-1000:].contiguous(), W))
    q = fp8_quantize(x)
    assert torch.equal(q.codes[-1000:], fp8_quantize(x[-1000:]).codes)
    del x, y, q
    x = torch.empty(70001, 32, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    W = fp8_quantize(torch.empty(31000, 32, device=DEV).normal_(generator=g), 128)
    y = fp8_linear(x, W)
    assert near(y[-200:], fp8_linear(x[-200:].contiguous(), W))


def test_runs_repeat_and_replay():
    """The same bits from another stream, and from captured graphs replayed on
    new inputs, for the one-launch and the two-launch forms and dW."""
    g = torch.Generator(device=DEV).manual_seed(3)
    W = fp8_quantize(torch.empty(300, 520, device=DEV).normal_(generator=g), 128)
    for M in (3, 40, 300):
        xs = [torch.empty(M, 520, dtype=torch.bfloat16, device=DEV).normal_(generator=g) for _ in range(3)]
        dy = torch.empty(M, 300, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
        run = lambda x: (fp8_linear(x, W), fp8_linear_dw(dy, x))  # noqa: E731
        want = [run(x) for x in xs]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = run(xs[0])
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(other, want[0]))
        x = xs[0].clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = run(x)
        for i in (0, 1, 2, 1):
            x.copy_(xs[i])
            run(xs[2])
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want[i]))


# --------------------------------------------------------------- checkpoints

def _close(got, want, slack):
    """bf16 of a value good to 2^-20, and `slack` absolute."""
    assert np.all(np.abs(host(got) - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -18) + slack)


@pytest.mark.parametrize("R,I", [(1, 16), (3, 32), (7, 48), (64, 2880), (130, 160), (1000, 96)])
@pytest.mark.parametrize("alpha,limit", [(1.702, 7.0), (1.0, 0.37), (-0.5, 1e4)])
def test_swiglu(R, I, alpha, limit):
    print("swiglu", R, I, alpha, limit, flush=True)
    r = np.random.default_rng(R + I)
    h = ref.bf16(r.normal(size=(R, 2 * I)) * limit * 0.7 if limit < 100 else r.normal(size=(R, 2 * I)) * 3)
    h[r.random(size=h.shape) < 0.05] = limit if ref.bf16([limit])[0] == np.float32(limit) else 0.0
    da = ref.bf16(r.normal(size=(R, I)))
    lim = float(np.float32(limit))
    a, c = swiglu_mxfp8(dev(h, torch.bfloat16), alpha, limit)
    codes, e = ref.swiglu_codes(h, lim)
    assert np.array_equal(c.codes.cpu().numpy(), codes)
    assert np.array_equal(c.scales.cpu().numpy(), (e + 127).astype(np.uint8))
    v = ref.values(codes, e, 1, 32)
    tiny = 2.0 ** -130
    _close(a, ref.swiglu(h.astype(np.float64), alpha, lim), tiny)
    dh, again = swiglu_mxfp8_backward(c, dev(da, torch.bfloat16))
    g = ref.swiglu_grad(v, da.astype(np.float64), alpha, lim)
    # 1 + alpha g (1 - s) cancels near its zero: fp32 steps of terms up to
    # |alpha g| s (1 - s) < 0.3 plus 1, times |da| (|u| + 1) s
    size = np.abs(da) * (np.abs(np.clip(v[:, 1::2], -lim, lim)) + 1)
    slack = np.zeros_like(g)
    slack[:, 0::2] = size * 2.0 ** -20 * (1 + np.abs(alpha * np.minimum(v[:, 0::2], lim)))
    _close(dh, g, slack + tiny)
    _close(again, ref.swiglu(v, alpha, lim), tiny)
    hr, ar = swiglu_mxfp8_restore(c)
    assert np.array_equal(host(hr), v) and torch.equal(ar, again)
    # what the checkpoint decides is what the forward decided
    assert np.array_equal(v[:, 0::2] > lim, h[:, 0::2] > lim)
    assert np.array_equal(np.abs(v[:, 1::2]) > lim, np.abs(h[:, 1::2]) > lim)
    assert swiglu_mxfp8(dev(h, torch.bfloat16), alpha, limit, activation=False)[0] is None
    assert swiglu_mxfp8_backward(c, dev(da, torch.bfloat16), activation=False)[1] is None


def test_swiglu_every_bf16_near_the_bounds():
    """All bf16 values in [6, 9] of both signs, as gates and as ups, beside
    block maxima that make the grid step 2^-4 .. 16."""
    bits = np.arange(0x40C0, 0x4110, dtype=np.uint32) << 16
    v = np.concatenate([bits.view(np.float32), -bits.view(np.float32)])
    h = np.zeros((9 * len(v), 32), np.float32)
    for j, top in enumerate([7.0, 10.0, 14.0, 30.0, 60.0, 120.0, 250.0, 500.0, 1000.0]):
        rows = slice(j * len(v), (j + 1) * len(v))
        h[rows, 0], h[rows, 3], h[rows, 31] = v, v, ref.bf16([top])[0]
    _, c = swiglu_mxfp8(dev(h, torch.bfloat16))
    codes, e = ref.swiglu_codes(h, 7.0)
    assert np.array_equal(c.codes.cpu().numpy(), codes)
    x = ref.values(codes, e, 1, 32)
    assert np.array_equal(x[:, 0] > 7, h[:, 0] > 7) and np.array_equal(np.abs(x[:, 3]) > 7, np.abs(h[:, 3]) > 7)


def test_swiglu_non_finite():
    h = np.zeros((6, 32), np.float32)
    h[0, 0], h[1, 1], h[2, 0], h[3, 0], h[4, 1], h[5, 1] = np.nan, np.nan, np.inf, -np.inf, np.inf, -np.inf
    h[:, 2] = 3.0
    a, c = swiglu_mxfp8(dev(h, torch.bfloat16))
    a = a.float().cpu().numpy()
    assert np.isnan(a[0, 0]) and np.isnan(a[1, 0]) and a[3, 0] == 0 and a[4, 0] == 0 and a[5, 0] == 0
    assert abs(a[2, 0] - 7.0) < 0.04
    _, e = ref.swiglu_codes(h, 7.0)
    assert np.array_equal(c.scales.cpu().numpy()[:, 0], (e + 127).astype(np.uint8)[:, 0])
    codes = c.codes.cpu().numpy()
    for i, j in enumerate([0, 1, 0, 0, 1, 1]):
        assert codes[i, j] & 0x7F == 0x7F and np.count_nonzero(codes[i]) == 2
    dh, again = swiglu_mxfp8_backward(c, torch.ones(6, 16, dtype=torch.bfloat16, device=DEV))
    dh = dh.float().cpu().numpy()
    assert np.all(dh[[0, 1, 2, 3, 4, 5], [0, 1, 0, 0, 1, 1]] == 0)
    assert torch.all(again[:, 0].isnan()) and torch.all(again[:, 1:].isfinite())


def test_swiglu_past_32_bits_and_replay():
    g = torch.Generator(device=DEV).manual_seed(0)
    h = torch.empty(400000, 5760, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    a, c = swiglu_mxfp8(h)
    at, ct = swiglu_mxfp8(h[-300:].contiguous())
    assert torch.equal(a[-300:], at) and torch.equal(c.codes[-300:], ct.codes) and torch.equal(c.scales[-300:], ct.scales)
    dh, _ = swiglu_mxfp8_backward(c, a)
    assert torch.equal(dh[-300:], swiglu_mxfp8_backward(ct, at)[0])
    del h, a, c, dh
    x = torch.empty(33, 640, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    y = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, c = swiglu_mxfp8(x)
        dh, again = swiglu_mxfp8_backward(c, a)
    for i in range(3):
        x.copy_(y * (i + 1))
        a2, c2 = swiglu_mxfp8(x.clone())
        d2, g2 = swiglu_mxfp8_backward(c2, a2)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, a2) and torch.equal(c.codes, c2.codes) and torch.equal(dh, d2) and torch.equal(again, g2)
