"""The norm without a GPU: refusals, and the reference's gradients against
differences."""
import numpy as np
import pytest
import torch

import norm_ref as ref
from mxfp4_weight_mixture_02_amd import ops, rms_norm, rms_norm_backward

FAKE = 0x10000   # never dereferenced: every call below returns from host checks
BIG = 1 << 60


def test_reference_gradient_against_differences():
    r = np.random.default_rng(0)
    s, w, dy, ds = r.normal(size=(3, 10)) * 2, r.normal(size=10), r.normal(size=(3, 10)), r.normal(size=(3, 10))
    eps = 1e-2
    _, rstd = ref.norm(s, w, eps)
    dx, dw, _, _ = ref.backward(s, rstd, w, dy, ds)

    def loss(s, w):
        return (ref.norm(s, w, eps)[0] * dy).sum() + (s * ds).sum()

    h = 1e-6   # differences are off by h^2 of a third derivative and 1e-16 / h of the loss
    for i in range(3):
        for j in range(10):
            d = np.zeros_like(s)
            d[i, j] = h
            assert abs((loss(s + d, w) - loss(s - d, w)) / (2 * h) - dx[i, j]) < 1e-7
    for j in range(10):
        d = np.zeros_like(w)
        d[j] = h
        assert abs((loss(s, w + d) - loss(s, w - d)) / (2 * h) - dw[j]) < 1e-7


def _refused(code, rc):
    assert rc == code and ops.lib().mxfp4_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(T=0), -1), (dict(H=0), -1), (dict(H=32769), -2), (dict(T=1 << 28, H=128), -2), (dict(T=1 << 40), -2),
    (dict(T=(1 << 28) - 15, H=1), -2), (dict(T=(1 << 26) + 4, H=300), -2), (dict(x=None), -1), (dict(w=None), -1), (dict(rstd=None), -1),
    (dict(y=None, codes=None, scales=None), -1), (dict(scales=None), -1), (dict(codes=None), -1), (dict(sum=None), -1),
    (dict(res=None), -1), (dict(dtype=2), -1), (dict(wt=7), -1), (dict(x=FAKE + 1), -1), (dict(dtype=0, res=FAKE + 2), -1),
    (dict(sum=FAKE + 1), -1), (dict(wt=0, w=FAKE + 2), -1), (dict(y=FAKE + 1), -1), (dict(codes=FAKE + 8), -1),
    (dict(rstd=FAKE + 2), -1), (dict(eps=0.0), -1), (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1),
    (dict(eps=float("inf")), -1)])
def test_forward_refuses(kw, code):
    d = dict(x=FAKE, res=FAKE, dtype=1, w=FAKE, wt=1, T=4, H=8, eps=1e-5, sum=FAKE, y=FAKE, codes=FAKE, scales=FAKE,
             rstd=FAKE)
    d.update(kw)
    _refused(code, ops.lib().mxmoe_rms_norm(*d.values(), None))


@pytest.mark.parametrize("kw,code", [
    (dict(T=0), -1), (dict(H=0), -1), (dict(H=32769), -2), (dict(T=1 << 40), -2), (dict(s=None), -1),
    (dict(rstd=None), -1), (dict(w=None), -1), (dict(dy=None), -1), (dict(dx=None), -1), (dict(dw=None), -1),
    (dict(dtype=3), -1), (dict(wt=2), -1), (dict(dtype=0, s=FAKE + 2), -1), (dict(dsum=FAKE + 1), -1),
    (dict(dy=FAKE + 1), -1), (dict(dw=FAKE + 2), -1), (dict(rstd=FAKE + 1), -1), (dict(ws=None), -3), (dict(n=16), -3),
    (dict(ws=FAKE + 8), -1)])
def test_backward_refuses(kw, code):
    d = dict(s=FAKE, rstd=FAKE, w=FAKE, wt=1, dy=FAKE, dsum=FAKE, dtype=1, T=4, H=8, dx=FAKE, dw=FAKE, ws=FAKE, n=BIG)
    d.update(kw)
    _refused(code, ops.lib().mxmoe_rms_norm_backward(*d.values(), None))


def test_workspace_query():
    f = ops.lib().mxmoe_rms_norm_backward_workspace_bytes
    assert f(1, 8) > 0 and f(5000, 2880) > 2880 * 4
    for sizes in [(0, 8), (4, 0), (4, 32769), (1 << 40, 8)]:
        assert f(*sizes) == 0


def test_binding_refuses():
    bf = torch.bfloat16
    x, w = torch.zeros(4, 32, dtype=bf), torch.zeros(32)
    for match, call in [
            ("2-D", lambda: rms_norm(x[0], w)),
            ("fp32 or bf16", lambda: rms_norm(x.half(), w)),
            ("fp32 or bf16", lambda: rms_norm(x, w.half())),
            ("weight", lambda: rms_norm(x, w[:31])),
            ("residual", lambda: rms_norm(x, w, residual=x.float())),
            ("residual", lambda: rms_norm(x, w, residual=x[:3])),
            ("one of bf16 and fp8", lambda: rms_norm(x, w, bf16=False)),
            ("CUDA tensor", lambda: rms_norm(x, w)),
            ("dy", lambda: rms_norm_backward(x.float(), x, torch.zeros(4), w)),
            ("dy", lambda: rms_norm_backward(x[:3], x, torch.zeros(4), w)),
            ("rstd", lambda: rms_norm_backward(x, x, torch.zeros(3), w)),
            ("dsum", lambda: rms_norm_backward(x, x, torch.zeros(4), w, dsum=x.float())),
            ("CUDA tensor", lambda: rms_norm_backward(x, x, torch.zeros(4), w))]:
        with pytest.raises(ValueError, match=match):
            call()
