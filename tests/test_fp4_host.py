"""4-bit products without a GPU: refusals, and the reference's layouts."""
import numpy as np
import pytest
import torch

import fp4_ref as ref
from mxfp4_weight_mixture_02_amd import (Fp4Matrix, fp4_linear, fp4_linear_dx, fp4_matmul, fp4_matrix, fp4_quantize, ops)

FAKE = 0x10000   # never dereferenced: every call below returns from host checks
BIG = 1 << 60


def test_reference_layouts():
    r = np.random.default_rng(0)
    s = r.integers(0, 255, size=(5, 11)).astype(np.uint8)
    o = ref.ordered(s)
    assert o.shape == (2, 4, 16, 2) and o.size == 2 * 8 * 16
    for row in range(5):
        for b in range(11):
            assert o[b // 8, b // 2 % 4, row, b % 2] == s[row, b]
    q = Fp4Matrix(torch.zeros(5, 176, dtype=torch.uint8), torch.from_numpy(np.ascontiguousarray(o)), 352)
    q.check_shapes()
    assert np.array_equal(ref.natural(q)[:, :11], s) and not ref.natural(q)[:, 11:].any()


def test_reference_exact_values():
    g = torch.Generator().manual_seed(0)
    x = ref.whole(9, 100, g, "cpu")
    c, s = ref.quantize(x.numpy())
    q = Fp4Matrix(torch.from_numpy(c), torch.from_numpy(np.ascontiguousarray(ref.ordered(s))), 100)
    assert np.array_equal(ref.values(q), x.double().numpy())


def _refused(code, rc):
    assert rc == code and ops.lib().mxfp4_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(rows=0), -1), (dict(K=0), -1), (dict(K=(1 << 22) + 1), -2), (dict(rows=1 << 27), -2),
    (dict(rows=1 << 26, K=1 << 10), -2), (dict(x=None), -1), (dict(codes=None), -1), (dict(scales=None), -1),
    (dict(dtype=2), -1), (dict(dtype=0, x=FAKE + 2), -1), (dict(dtype=1, x=FAKE + 1), -1), (dict(codes=FAKE + 8), -1),
    (dict(scales=FAKE + 8), -1)])
def test_quantize_refuses(kw, code):
    d = dict(x=FAKE, dtype=1, rows=4, K=8, codes=FAKE, scales=FAKE)
    d.update(kw)
    _refused(code, ops.lib().mxmoe_fp4_quantize(*d.values(), None))


@pytest.mark.parametrize("kw,code", [
    (dict(rows=0), -1), (dict(K=0), -1), (dict(K=40), -2), (dict(rows=1 << 27), -2), (dict(s=None), -1),
    (dict(o=None), -1), (dict(o=FAKE + 8), -1)])
def test_scales_refuse(kw, code):
    d = dict(s=FAKE, rows=4, K=64, o=FAKE)
    d.update(kw)
    _refused(code, ops.lib().mxmoe_fp4_scales(*d.values(), None))


SIZES = [(dict(M=0), -1), (dict(N=0), -1), (dict(K=0), -1), (dict(M=1 << 27), -2), (dict(M=1 << 26, N=1 << 26), -2),
         (dict(wp=0), -1), (dict(wp=48), -1), (dict(K=40, wp=20), -1), (dict(w=None), -1), (dict(sw=None), -1),
         (dict(out=None), -1), (dict(out=FAKE + 4), -1), (dict(od=3), -1), (dict(w=FAKE + 8), -1),
         (dict(sw=FAKE + 8), -1), (dict(ws=None), -3), (dict(ws=FAKE + 8), -1)]


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(K=(1 << 22) + 1), -2), (dict(x=None), -1), (dict(sx=None), -1), (dict(x=FAKE + 8), -1), (dict(sx=FAKE + 8), -1),
    (dict(bias=FAKE + 1), -1), (dict(M=1, N=(1 << 27) - 15), -2)])
def test_matmul_refuses(kw, code):
    d = dict(M=4, N=4, K=64, x=FAKE, sx=FAKE, w=FAKE, wp=32, sw=FAKE, bias=None, od=1, out=FAKE, ws=FAKE, n=BIG)
    d.update(kw)
    _refused(code, ops.lib().mxmoe_fp4_matmul(*d.values(), None))


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(K=(1 << 22) + 1), -2), (dict(x=None), -1), (dict(x=FAKE + 1), -1), (dict(bias=FAKE + 1), -1), (dict(n=16), -3),
    (dict(M=16, N=(1 << 27) - 1), -2)])
def test_linear_refuses(kw, code):
    d = dict(M=4, N=4, K=64, x=FAKE, w=FAKE, wp=128, sw=FAKE, bias=None, od=1, out=FAKE, ws=FAKE, n=BIG)
    d.update(kw)
    _refused(code, ops.lib().mxmoe_fp4_linear(*d.values(), None))


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(K=(1 << 22) + 1), -2), (dict(N=(1 << 22) + 1), -2), (dict(dy=None), -1), (dict(dy=FAKE + 1), -1),
    (dict(n=128), -3), (dict(M=2000, n=1024), -3), (dict(M=1 << 26, N=1024), -2)])
def test_linear_dx_refuses(kw, code):
    d = dict(M=4, N=4, K=64, dy=FAKE, w=FAKE, wp=128, sw=FAKE, od=1, out=FAKE, ws=FAKE, n=BIG)
    d.update(kw)
    _refused(code, ops.lib().mxmoe_fp4_linear_dx(*d.values(), None))


def test_workspace_queries_refuse():
    L = ops.lib()
    fs = (L.mxmoe_fp4_matmul_workspace_bytes, L.mxmoe_fp4_linear_workspace_bytes, L.mxmoe_fp4_linear_dx_workspace_bytes)
    for f in fs:
        assert f(40, 4, 64, 0) > 0 and f(4, 4, 7, 1) > 0
        for sizes in [(0, 4, 64), (4, 0, 64), (4, 4, 0), (4, 4, 1 << 23), (1 << 27, 4, 4)]:
            assert f(*sizes, 1) == 0
        assert f(4, 4, 64, 2) == 0


def test_binding_refuses():
    bf, u8 = torch.bfloat16, torch.uint8
    x = torch.zeros(4, 64, dtype=bf)
    w, q = Fp4Matrix.empty(8, 64, "cpu"), Fp4Matrix.empty(4, 64, "cpu")
    flat = Fp4Matrix(torch.zeros(8, 32, dtype=u8), w.scales, 64)
    flat.check_shapes()
    for match, call in [
            ("at least one", lambda: Fp4Matrix.empty(0, 32, "cpu")),
            ("fp32 or bf16", lambda: fp4_quantize(x.half())),
            ("2-D", lambda: fp4_quantize(x[0])),
            ("CUDA tensor", lambda: fp4_quantize(x)),
            ("K a multiple of 32", lambda: fp4_matrix(torch.zeros(4, 20, dtype=u8), torch.zeros(4, 1, dtype=u8))),
            ("scales", lambda: fp4_matrix(torch.zeros(4, 32, dtype=u8), torch.zeros(4, 1, dtype=u8))),
            ("codes", lambda: fp4_matrix(torch.zeros(4, 32), torch.zeros(4, 2, dtype=u8))),
            ("CUDA tensor", lambda: fp4_matrix(torch.zeros(4, 32, dtype=u8), torch.zeros(4, 2, dtype=u8))),
            ("padded", lambda: fp4_matmul(flat, w)),
            ("do not hold", lambda: fp4_matmul(q, Fp4Matrix(w.codes[:, :16].contiguous(), w.scales, 64))),
            ("do not hold", lambda: fp4_linear(x, Fp4Matrix(torch.zeros(8, 20, dtype=u8), w.scales, 40))),
            ("w.scales", lambda: fp4_matmul(q, Fp4Matrix(w.codes, w.scales[:, :3], 64))),
            ("K=64, w K=32", lambda: fp4_matmul(q, Fp4Matrix.empty(8, 32, "cpu"))),
            ("bias", lambda: fp4_matmul(q, w, bias=torch.zeros(8))),
            ("CUDA tensor", lambda: fp4_matmul(q, w)),
            ("expected", lambda: fp4_linear(x.float(), w)),
            ("expected", lambda: fp4_linear(x[:, :32], w)),
            ("CUDA tensor", lambda: fp4_linear(x, w)),
            ("expected", lambda: fp4_linear_dx(x, w)),
            ("CUDA tensor", lambda: fp4_linear_dx(torch.zeros(4, 8, dtype=bf), w))]:
        with pytest.raises(ValueError, match=match):
            call()
