"""The norm on the GPU against float64: every split of a row over waves, types,
alignments, extreme rows, both results, gradients, graphs and streams."""
import numpy as np
import pytest
import torch

import fp8_ref
import norm_ref as ref
from gpu_helpers import to_f64
from mxfp4_weight_mixture_02_amd import fp8_matmul, fp8_quantize, ops, rms_norm, rms_norm_backward

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
# A row's sums pass through at most 48 additions in a lane, 6 over the wave
# and 15 over the waves: below 2^-24 * 72 < 2^-17 of the magnitudes summed.
SUM = 2.0 ** -17
BF16 = 2.0 ** -8          # half a step, relative
TINY = 2.0 ** -133        # a step of bf16's subnormals

# rows x columns: one wave a row in 2, 4 and 6 chunks, four waves in 1, 2 and
# 4, sixteen in 2 and 4; one element, odd sizes, whole and broken blocks
SIZES = [(1, 1), (3, 7), (5, 128), (2, 130), (1030, 40), (1025, 513), (1026, 1030), (1027, 2880), (700, 2880), (37, 96),
         (3, 2049), (3, 5000), (2, 8192), (2, 9000), (2, 16384), (2, 20000), (1, 32768), (3, 32767)]


def _np(t):
    return None if t is None else to_f64(t)


def _draw(T, H, f32, w32, res, seed=0, shift=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    t = torch.float32 if f32 else torch.bfloat16

    def normal(n, std, dt):
        # `shift` elements into an allocation: rows that are not 16-byte aligned
        flat = torch.empty(n[0] * n[1] + shift, dtype=dt, device=DEV)
        v = flat[shift:].view(n)
        v.copy_(torch.randn(n, generator=g, device=DEV) * std)
        return v

    x = normal((T, H), 1.5, t)
    r = normal((T, H), 2.0, t) if res else None
    w = normal((1, H), 1.0, torch.float32 if w32 else torch.bfloat16)[0]
    dy = normal((T, H), 0.5, torch.bfloat16)
    ds = normal((T, H), 0.3, t) if res else None
    return x, r, w, dy, ds


def _check_codes(q, y, T, H):
    """Scales: the smallest that hold the block; elements within half a step."""
    Hp = -(-H // 128) * 128
    e = q.scales[:, :T].cpu().numpy().astype(np.int64).T - 127
    codes = q.codes.cpu().numpy()
    assert not codes[:, H:].any()
    p = np.zeros((T, Hp))
    p[:, :H] = y
    b = p.reshape(T, -1, 128)
    top = np.abs(b).max(2)
    assert np.all(top * (1 - SUM) <= np.ldexp(448.0, e))
    assert np.all((np.ldexp(448.0, e - 1) < top * (1 + SUM)) | (e == -127))
    got = fp8_ref.values(codes, e, 1, 128).reshape(b.shape)
    # half a step: 2^-4 of a value, 2^-10 of the scale below its 2^-6
    tol = np.maximum(np.abs(b) * 2.0 ** -4, np.ldexp(1.0, e)[:, :, None] * 2.0 ** -10) + np.abs(b) * SUM
    assert np.all(np.abs(got - b) <= tol)


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("f32,w32,res,shift", [(0, 1, 1, 0), (1, 0, 0, 0), (1, 1, 1, 1), (0, 0, 0, 1)])
def test_forward(T, H, f32, w32, res, shift):
    print("norm", T, H, f32, w32, res, shift, flush=True)
    x, r, w, _, _ = _draw(T, H, f32, w32, res, shift=shift)
    n = rms_norm(x, w, residual=r, eps=1e-5, fp8=True)
    s = ref.stream(_np(x), _np(r), f32)
    assert np.array_equal(_np(n.sum), s) and (n.sum is x) == (not res)
    y, rstd = ref.norm(s, _np(w), 1e-5)
    assert np.all(np.abs(_np(n.rstd) - rstd) <= rstd * SUM)
    assert np.all(np.abs(_np(n.y) - y) <= np.abs(y) * (BF16 + 2 * SUM) + TINY)
    _check_codes(n.y8, y, T, H)
    # either result alone has the same bits
    a, b = rms_norm(x, w, residual=r, eps=1e-5), rms_norm(x, w, residual=r, eps=1e-5, bf16=False, fp8=True)
    assert a.y8 is None and b.y is None
    assert torch.equal(a.y, n.y) and torch.equal(b.y8.codes, n.y8.codes)
    assert torch.equal(b.y8.scales[:, :T], n.y8.scales[:, :T])


@pytest.mark.parametrize("T,H", SIZES + [(5000, 96), (4099, 2880)])
@pytest.mark.parametrize("f32,w32,res,shift", [(0, 1, 1, 0), (1, 0, 0, 0), (1, 1, 1, 1), (0, 0, 0, 1)])
def test_backward(T, H, f32, w32, res, shift):
    print("norm gradient", T, H, f32, w32, res, shift, flush=True)
    x, _, w, dy, ds = _draw(T, H, f32, w32, res, seed=1, shift=shift)
    rstd = rms_norm(x, w).rstd
    dx, dw = rms_norm_backward(dy, x, rstd, w, dsum=ds)
    wx, ww, size, wsize = ref.backward(_np(x), _np(rstd), _np(w), _np(dy), _np(ds))
    half = 2.0 ** -24 if f32 else BF16
    assert dx.dtype == x.dtype and dw.dtype == torch.float32
    assert np.all(np.abs(_np(dx) - wx) <= np.abs(wx) * half + size * SUM + TINY)
    # dw: at most 5 rows a lane, 4 rows of a wave, 4 waves, 64 parts a slice, 16 slices: fewer than 128 additions, 2^-17
    assert np.all(np.abs(_np(dw) - ww) <= wsize * SUM)
    again = rms_norm_backward(dy, x, rstd, w, dsum=ds)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


@pytest.mark.parametrize("T,H", [(1100, 200), (6, 200), (6, 9000)])
def test_extreme_rows(T, H):
    """Rows whose squares fp32 does not hold, zeros, infinities and NaN: each
    keeps to itself."""
    x, _, w, dy, _ = _draw(T, H, 1, 1, 0)
    x[0] *= 1e30
    x[1] *= 1e-30
    x[2] = 0
    x[3, 5] = torch.nan
    x[4, 7] = torch.inf
    n = rms_norm(x, w, eps=1e-38, fp8=True)
    s = _np(x)
    with np.errstate(invalid="ignore"):
        y, rstd = ref.norm(s, _np(w), 1e-38)
    ok = [i for i in range(T) if i not in (3, 4)]
    assert np.all(np.abs(_np(n.rstd)[ok] - rstd[ok]) <= rstd[ok] * SUM)
    assert np.all(np.abs(_np(n.y)[ok] - y[ok]) <= np.abs(y[ok]) * (BF16 + 2 * SUM))
    assert torch.isnan(n.y[3]).all() and torch.isnan(n.y[4, 7]) and torch.all(n.y[4, :7] == 0)
    q = n.y8
    assert torch.all(q.codes[3, :H] & 0x7F == 0x7F) and torch.all(q.codes[3, H:] == 0) and q.codes[4, 7] & 0x7F == 0x7F
    keep = torch.tensor(ok, device=DEV)
    back = fp8_quantize(rms_norm(x[keep].contiguous(), w, eps=1e-38).y.float())
    # the same rows elsewhere: as the bf16 result's own codes, to its rounding
    d = (fp8_ref.values(q.codes[keep].cpu().numpy(), q.scales[:, keep].cpu().numpy().astype(int).T - 127, 1, 128) -
         fp8_ref.values(back.codes.cpu().numpy(), back.scales[:, :len(ok)].cpu().numpy().astype(int).T - 127, 1, 128))
    assert np.all(np.abs(d[:, :H]) <= np.abs(y[ok]) * 2.0 ** -3 * 1.1 + np.abs(y[ok]).max() * 2.0 ** -16)
    dx, dw = rms_norm_backward(dy, x, n.rstd, w)
    wx, _, size, _ = ref.backward(s[ok], _np(n.rstd)[ok], _np(w), _np(dy)[ok])
    assert np.all(np.abs(_np(dx)[ok] - wx) <= np.abs(wx) * 2.0 ** -24 + size * SUM + 2.0 ** -149)
    assert torch.isnan(dx[3]).all() and torch.isnan(dw).all()


@pytest.mark.parametrize("T,H", [(3, 100), (1029, 2880), (5, 4100)])
def test_nothing_else_is_written(T, H):
    """Outputs inside larger buffers; dx over dsum, sum over the residual."""
    x, r, w, dy, ds = _draw(T, H, 0, 1, 1)
    Hp, G = -(-H // 128) * 128, 64
    n = rms_norm(x, w, residual=r, fp8=True)

    def guarded(like):
        flat = torch.full((like.numel() + 2 * G,), 7, dtype=like.dtype, device=DEV)
        return flat, flat[G:-G].view(like.shape)

    (fy, y), (fc, c), (fr, rstd) = guarded(n.y), guarded(n.y8.codes), guarded(n.rstd)
    sc = torch.full((Hp // 128, -(-T // 16) * 16), 7, dtype=torch.uint8, device=DEV)
    total = r.clone()
    L, s = ops.lib(), torch.cuda.current_stream().cuda_stream
    p = lambda t: t.data_ptr()  # noqa: E731
    assert L.mxmoe_rms_norm(p(x), p(total), 1, p(w), 0, T, H, 1e-5, p(total), p(y), p(c), p(sc), p(rstd), s) == 0
    assert torch.equal(total, n.sum) and torch.equal(y, n.y) and torch.equal(c, n.y8.codes) and torch.equal(rstd, n.rstd)
    assert torch.equal(sc[:, :T], n.y8.scales[:, :T]) and torch.all(sc[:, T:] == 7)
    for f in (fy, fc, fr):
        assert torch.all(f[:G] == 7) and torch.all(f[-G:] == 7)
    dx, dw = rms_norm_backward(dy, n.sum, n.rstd, w, dsum=ds)
    (fd, d), (fw, w2) = guarded(ds), guarded(dw)
    d.copy_(ds)
    m = L.mxmoe_rms_norm_backward_workspace_bytes(T, H)
    ws = torch.empty(m, dtype=torch.uint8, device=DEV)
    assert L.mxmoe_rms_norm_backward(p(n.sum), p(n.rstd), p(w), 0, p(dy), p(d), 1, T, H, p(d), p(w2), p(ws), m, s) == 0
    assert torch.equal(d, dx) and torch.equal(w2, dw)
    for f in (fd, fw):
        assert torch.all(f[:G] == 7) and torch.all(f[-G:] == 7)


def test_rows_do_not_depend_on_the_others():
    """A row's bits are the same in any batch of the same split over waves."""
    x, r, w, _, _ = _draw(1500, 2880, 0, 1, 1)
    n = rms_norm(x, w, residual=r, fp8=True)
    m = rms_norm(x[100:1300].contiguous(), w, residual=r[100:1300].contiguous(), fp8=True)
    assert torch.equal(n.y[100:1300], m.y) and torch.equal(n.y8.codes[100:1300], m.y8.codes)
    assert torch.equal(n.y8.scales[:, 100:1300], m.y8.scales[:, :1200])


def test_result_feeds_an_8_bit_product():
    x, _, w, _, _ = _draw(33, 320, 0, 1, 0)
    n = rms_norm(x, w, fp8=True)
    wq = fp8_quantize(torch.randn(48, 320, device=DEV), 128)
    got = fp8_matmul(n.y8, wq, dtype=torch.float32)
    e = n.y8.scales[:, :33].cpu().numpy().astype(int).T - 127
    we = wq.scales.cpu().numpy().astype(int).T - 127
    a = fp8_ref.values(n.y8.codes.cpu().numpy(), e, 1, 128)
    b = fp8_ref.values(wq.codes.cpu().numpy(), we, 128, 128)
    assert np.all(np.abs(to_f64(got) - a @ b.T) <= np.abs(a) @ np.abs(b).T * 384 * 2.0 ** -24)


@pytest.mark.parametrize("T,H", [(1, 2880), (1300, 320)])
def test_captured(T, H):
    """Two graphs replayed in turn, with eager calls between, on a stream of
    their own, give the eager bits."""
    sets = [_draw(T, H, 0, 1, 1, seed=i) for i in range(3)]

    def step(x, r, w, dy, ds):
        n = rms_norm(x, w, residual=r, fp8=True)
        return (n.y, n.y8.codes, n.rstd, n.sum) + rms_norm_backward(dy, n.sum, n.rstd, w, dsum=ds)

    want = [step(*v) for v in sets]
    hold = [[t.clone() for t in sets[0]] for _ in range(2)]
    side = torch.cuda.Stream()
    graphs, outs = [], []
    for h in hold:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(step(*h))
        graphs.append(g)
    for i in range(4):
        for h, j in zip(hold, (i % 3, (i + 1) % 3)):
            for a, b in zip(h, sets[j]):
                a.copy_(b)
        step(*sets[2])
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for o, j in zip(outs, (i % 3, (i + 1) % 3)):
            assert all(torch.equal(a, b) for a, b in zip(o, want[j]))
