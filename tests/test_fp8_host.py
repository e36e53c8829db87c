"""8-bit products and checkpoints without a GPU: refusals, and the reference
against the oracle's MXFP8 and closed forms."""
import numpy as np
import pytest
import torch

import fp8_ref as ref
from mxfp4_weight_mixture_02_amd import (Fp8Matrix, SwigluCheckpoint, fp8_linear, fp8_linear_dw, fp8_matmul,
                                         fp8_quantize, fp8_quantize_t, fp8_transpose, ops, swiglu_mxfp8,
                                         swiglu_mxfp8_backward)
from oracle import mxfp8

FAKE = 0x10000   # never dereferenced: every call below returns from host checks
BIG = 1 << 40


def test_reference_quantizer_is_the_oracles_at_blocks_of_32():
    r = np.random.default_rng(0)
    x = r.normal(size=(7, 96)) * np.exp(r.normal(size=(7, 96)) * 5)
    c, e, _ = ref.quantize(x, 1, 32)
    oc, os_ = mxfp8.quantize(x)
    assert np.array_equal(c, oc) and np.array_equal(e + 127, os_)


def test_reference_clamp_sides():
    """7.2 rounds to 7.0 at its block's step of 0.5 and is moved back above
    the bound; 7.0 stays on it; an up of -7.2 likewise, a gate of -7.2 not."""
    h = np.zeros((1, 32))
    h[0, :6] = [7.2, 7.2, 7.0, -7.2, -7.2, 6.8]
    c, e = ref.swiglu_codes(h, 7.0)
    assert ref.values(c, e, 1, 32)[0, :6].tolist() == [7.5, 7.5, 7.0, -7.5, -7.0, 7.0]


def test_reference_gradient_against_differences():
    r = np.random.default_rng(1)
    h, da = r.normal(size=(3, 32)) * 4, r.normal(size=(3, 16))
    g = ref.swiglu_grad(h, da, 1.702, 7.0)
    for i in range(32):
        d = np.zeros((3, 32))
        d[:, i] = 1e-6
        num = ((ref.swiglu(h + d, 1.702, 7.0) - ref.swiglu(h - d, 1.702, 7.0)) * da).sum(1) / 2e-6
        # rounding 1e-15 * |a| / 1e-6 with |a| <= 56 |da|, truncation 1e-12 of a third derivative
        assert np.abs(num - g[:, i]).max() < 1e-6


def _refused(code, rc):
    assert rc == code and ops.lib().mxfp4_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(rows=0), -1), (dict(K=0), -1), (dict(K=(1 << 22) + 1), -2), (dict(rows=1 << 27), -2),
    (dict(rows=1 << 26, K=1 << 12), -2), (dict(x=None), -1), (dict(codes=None), -1), (dict(scales=None), -1),
    (dict(dtype=2), -1), (dict(dtype=0, x=FAKE + 2), -1), (dict(dtype=1, x=FAKE + 1), -1),
    (dict(block_rows=2), -1), (dict(codes=FAKE + 8), -1), (dict(scales=FAKE + 8), -1)])
def test_quantize_refuses(kw, code):
    d = dict(x=FAKE, dtype=1, rows=4, K=8, block_rows=1, codes=FAKE, scales=FAKE)
    d.update(kw)
    _refused(code, ops.lib().mxmoe_fp8_quantize(*d.values(), None))
    if "block_rows" not in kw and "K" not in kw and "rows" not in kw:
        d.pop("block_rows")
        _refused(code, ops.lib().mxmoe_fp8_quantize_t(*d.values(), None))


def test_transpose_refuses():
    f = ops.lib().mxmoe_fp8_transpose
    _refused(-1, f(FAKE, FAKE, 0, 8, FAKE, FAKE, None))
    _refused(-2, f(FAKE, FAKE, (1 << 22) + 1, 8, FAKE, FAKE, None))
    _refused(-1, f(FAKE, FAKE, 8, 8, None, FAKE, None))
    _refused(-1, f(FAKE, FAKE, 8, 8, FAKE + 4, FAKE, None))


@pytest.mark.parametrize("kw,code", [
    (dict(M=0), -1), (dict(N=0), -1), (dict(K=0), -1), (dict(K=(1 << 22) + 1), -2), (dict(M=1 << 27), -2),
    (dict(M=1 << 26, N=1 << 26), -2), (dict(x=None), -1), (dict(sw=None), -1), (dict(out=None), -1),
    (dict(br=64), -1), (dict(od=3), -1), (dict(out=FAKE + 4), -1), (dict(bias=FAKE + 1), -1),
    (dict(br=1, sw=FAKE + 1), -1), (dict(w=FAKE + 8), -1), (dict(ws=None), -3), (dict(ws=FAKE + 8), -1),
    (dict(M=128, N=256, K=4096, n=1 << 16), -3)])
def test_matmul_refuses(kw, code):
    d = dict(M=4, N=4, K=8, x=FAKE, sx=FAKE, w=FAKE, sw=FAKE, br=128, bias=None, od=1, out=FAKE, ws=FAKE, n=BIG)
    d.update(kw)
    _refused(code, ops.lib().mxmoe_fp8_matmul(*d.values(), None))


@pytest.mark.parametrize("kw,code", [
    (dict(M=0), -1), (dict(K=(1 << 22) + 1), -2), (dict(x=None), -1), (dict(x=FAKE + 1), -1), (dict(w=None), -1),
    (dict(out=FAKE + 4), -1), (dict(od=7), -1), (dict(ws=None), -3), (dict(n=16), -3), (dict(ws=FAKE + 8), -1)])
def test_linear_refuses(kw, code):
    d = dict(M=4, N=4, K=8, x=FAKE, w=FAKE, sw=FAKE, bias=None, od=1, out=FAKE, ws=FAKE, n=BIG)
    d.update(kw)
    _refused(code, ops.lib().mxmoe_fp8_linear(*d.values(), None))


@pytest.mark.parametrize("kw,code", [
    (dict(M=0), -1), (dict(M=(1 << 22) + 1), -2), (dict(dy=None), -1), (dict(dw=FAKE + 4), -1),
    (dict(x=FAKE + 1), -1), (dict(ws=None), -3), (dict(n=256), -3), (dict(ws=FAKE + 8), -1)])
def test_linear_dw_refuses(kw, code):
    d = dict(M=4, N=4, K=8, dy=FAKE, x=FAKE, dw=FAKE, ws=FAKE, n=BIG)
    d.update(kw)
    _refused(code, ops.lib().mxmoe_fp8_linear_dw(*d.values(), None))


def test_workspace_queries_refuse():
    L = ops.lib()
    assert L.mxmoe_fp8_matmul_workspace_bytes(4, 4, 8, 0) > 0 and L.mxmoe_fp8_linear_workspace_bytes(4, 4, 8, 1) > 0
    for sizes in [(0, 4, 8), (4, 0, 8), (4, 4, 0), (4, 4, 1 << 23)]:
        assert L.mxmoe_fp8_matmul_workspace_bytes(*sizes, 1) == 0
        assert L.mxmoe_fp8_linear_workspace_bytes(*sizes, 1) == 0
    assert L.mxmoe_fp8_linear_dw_workspace_bytes(1 << 23, 4, 4) == 0
    assert L.mxmoe_fp8_matmul_workspace_bytes(4, 4, 8, 2) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(R=0), -1), (dict(I=0), -1), (dict(I=24), -2), (dict(R=1 << 30, I=16), -2), (dict(R=1 << 22, I=1 << 12), -2),
    (dict(alpha=float("nan")), -1), (dict(limit=float("inf")), -1), (dict(limit=0.0), -1), (dict(limit=-7.0), -1)])
def test_swiglu_refuses(kw, code):
    d = dict(R=4, I=32, alpha=1.702, limit=7.0)
    d.update(kw)
    n = d.values()
    L = ops.lib()
    _refused(code, L.mxmoe_swiglu8_forward(FAKE, *n, FAKE, FAKE, FAKE, None))
    _refused(code, L.mxmoe_swiglu8_backward(FAKE, FAKE, FAKE, *n, FAKE, FAKE, None))
    _refused(code, L.mxmoe_swiglu8_restore(FAKE, FAKE, *n, FAKE, FAKE, None))


def test_swiglu_refuses_pointers():
    L, n = ops.lib(), (4, 32, 1.702, 7.0)
    _refused(-1, L.mxmoe_swiglu8_forward(None, *n, FAKE, FAKE, FAKE, None))
    _refused(-1, L.mxmoe_swiglu8_forward(FAKE + 8, *n, FAKE, FAKE, FAKE, None))
    _refused(-1, L.mxmoe_swiglu8_backward(FAKE, FAKE, None, *n, FAKE, FAKE, None))
    _refused(-1, L.mxmoe_swiglu8_backward(FAKE, FAKE, FAKE, *n, FAKE, FAKE + 2, None))
    _refused(-1, L.mxmoe_swiglu8_restore(FAKE, FAKE, *n, None, None, None))


def test_binding_refuses():
    bf = torch.bfloat16
    x = torch.zeros(4, 32, dtype=bf)
    w = Fp8Matrix.empty(8, 32, 128, "cpu")
    q = Fp8Matrix.empty(4, 32, 1, "cpu")
    for match, call in [
            ("block_rows", lambda: Fp8Matrix.empty(4, 32, 64, "cpu")),
            ("at least one", lambda: Fp8Matrix.empty(0, 32, 1, "cpu")),
            ("fp32 or bf16", lambda: fp8_quantize(x.half())),
            ("2-D", lambda: fp8_quantize(x[0])),
            ("CUDA tensor", lambda: fp8_quantize(x)),
            ("2-D", lambda: fp8_quantize_t(x[0])),
            ("block_rows 128", lambda: fp8_transpose(q)),
            ("x needs block_rows 1", lambda: fp8_matmul(w, w)),
            ("K=32, w K=64", lambda: fp8_matmul(q, Fp8Matrix.empty(8, 64, 128, "cpu"))),
            ("bias", lambda: fp8_matmul(q, w, bias=torch.zeros(8))),
            ("w.scales", lambda: fp8_matmul(q, Fp8Matrix(w.codes, w.scales[:, :0], 32, 128))),
            ("w.codes", lambda: fp8_matmul(q, Fp8Matrix(w.codes, w.scales, 200, 128))),
            ("CUDA tensor", lambda: fp8_matmul(q, w)),
            ("expected", lambda: fp8_linear(x.float(), w)),
            ("expected", lambda: fp8_linear(x[:, :16], w)),
            ("block_rows 128", lambda: fp8_linear(x, q)),
            ("CUDA tensor", lambda: fp8_linear(x, w)),
            ("expected", lambda: fp8_linear_dw(x, x[:2])),
            ("CUDA tensor", lambda: fp8_linear_dw(x, x)),
            ("2I a multiple of 32", lambda: swiglu_mxfp8(x[:, :24])),
            ("expected", lambda: swiglu_mxfp8(x.float())),
            ("CUDA tensor", lambda: swiglu_mxfp8(x)),
            ("scales", lambda: swiglu_mxfp8_backward(
                SwigluCheckpoint(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)), x)),
            ("da", lambda: swiglu_mxfp8_backward(
                SwigluCheckpoint(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 1, dtype=torch.uint8)), x))]:
        with pytest.raises(ValueError, match=match):
            call()
