"""The balance losses' sums over tokens do not overflow before the mean."""
import numpy as np
import pytest
import torch

from mxfp4_weight_mixture_02_amd import moe_balance

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("T", [33, 200, 3001, (1 << 18) + 5])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("cut", [None, 7])
def test_a_square_beyond_fp32_has_a_finite_mean(T, score, cut):
    """One logit of 3e19, whose square is no fp32: the mean over the tokens is."""
    print("squares", T, score, cut, flush=True)
    x = torch.zeros(T, 4, device=DEV)
    x[5, 2] = 3e19
    idx = torch.zeros(T, 1, dtype=torch.int32, device=DEV)
    offsets = None if cut is None else torch.tensor([0, cut, T], dtype=torch.int32, device=DEV)
    got = float(moe_balance(x, idx, score=score, offsets=offsets).losses[1])
    # the other tokens' squares, log(4)^2, are far below a step of it; one rounding to fp32
    want = float(np.float32(3e19)) ** 2 / T
    assert abs(got - want) <= want * 2.0 ** -23
