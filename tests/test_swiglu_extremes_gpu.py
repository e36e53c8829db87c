"""The SwiGLU checkpoint and its backward pass at the ends of bf16's range,
where alpha times the gate is no finite float."""
import numpy as np
import pytest
import torch

import fp8_ref as ref
from mxfp4_weight_mixture_02_amd import swiglu_mxfp8, swiglu_mxfp8_backward, swiglu_mxfp8_restore

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def bf(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(DEV).bfloat16()


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("alpha", [1.702, -1.702, 30.0, -30.0, 1e30, 0.0])
@pytest.mark.parametrize("limit", [7.0, 3.0e38])
def test_gates_far_from_zero(alpha, limit):
    """A gate whose sigmoid is 0 has no gradient, one whose sigmoid is 1 that
    of the identity, however large alpha times it is."""
    print("swiglu extremes", alpha, limit, flush=True)
    gates = [s * v for v in (1e4, 1e30, 1e37, 1.1e38, 2.5e38, 3.0e38) for s in (1.0, -1.0)]
    h = np.zeros((len(gates), 32), np.float32)
    h[:, 0], h[:, 1], h[:, 2], h[:, 3] = gates, -0.5, 1.0, 0.25
    h = ref.bf16(h)
    da = ref.bf16(np.full((len(gates), 16), 0.5))
    a, c = swiglu_mxfp8(bf(h), alpha, limit)
    v = ref.values(c.codes.cpu().numpy(), c.scales.cpu().numpy().astype(np.int64) - 127, 1, 32)
    dh, again = swiglu_mxfp8_backward(c, bf(da))
    lim, al = float(np.float32(limit)), float(np.float32(alpha))
    # bf16 (2^-8) of an fp32 value whose exponential and reciprocal are good to 2^-20;
    # gates here are 0 or so large that no sigmoid is between 0 and 1
    for got, want in ((a, ref.swiglu(h.astype(np.float64), al, lim)), (again, ref.swiglu(v, al, lim)),
                      (dh, ref.swiglu_grad(v, da.astype(np.float64), al, lim))):
        assert torch.all(got.isfinite())
        assert np.all(np.abs(host(got) - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -18) + 2.0 ** -130)


def test_largest_values():
    """bf16's largest values round to 2^128, beyond fp32: restored as
    infinities on their own side of every bound, and no gradient is NaN."""
    top = float(torch.finfo(torch.bfloat16).max)
    h = np.zeros((4, 32), np.float32)
    h[0, 0], h[1, 0], h[2, 1], h[3, 1] = top, -top, top, -top
    a, c = swiglu_mxfp8(bf(h))
    hr, ar = swiglu_mxfp8_restore(c)
    dh, again = swiglu_mxfp8_backward(c, bf(np.ones((4, 16))))
    assert host(hr)[[0, 1, 2, 3], [0, 0, 1, 1]].tolist() == [np.inf, -np.inf, np.inf, -np.inf]
    for t in (a, ar, dh, again):
        assert torch.all(t.isfinite())
    assert torch.equal(a, again) and torch.equal(a, ar)
    assert np.all(host(dh)[[0, 1, 2, 3], [0, 0, 1, 1]] == 0)
