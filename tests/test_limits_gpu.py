"""The last sizes that an entry point takes."""
import pytest
import torch

from mxfp4_weight_mixture_02_amd import RouteOptions, moe_route, moe_route_backward

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_most_tokens_of_a_routing():
    """2^26 - 1 tokens of two experts, k = 1: the gradient of one token a wave
    has 64 threads a token, and a launch 2^32 - 1."""
    T, o = (1 << 26) - 1, RouteOptions(renorm=False)
    g = torch.Generator(device=DEV).manual_seed(0)
    x = torch.randn(T, 2, generator=g, device=DEV)
    r = moe_route(x, 1, o)
    z = x[:, 1].double() - x[:, 0].double()
    # chosen by the scores' fp32 values, equal ones by the index
    idx = (torch.sigmoid(z).float() > torch.sigmoid(-z).float()).int()
    assert torch.equal(r.topk_idx[:, 0], idx)
    n = int(idx.sum())
    assert r.expert_offsets.tolist() == [0, T - n, T]
    assert torch.equal(r.sorted_rows[:T - n].long(), (idx == 0).nonzero()[:, 0])
    assert torch.equal(r.sorted_rows[T - n:].long(), (idx == 1).nonzero()[:, 0])
    dw = torch.randn(T, 1, generator=g, device=DEV)
    d = moe_route_backward(x, r.topk_idx, dw, o)
    # w = sigmoid(l_chosen - l_other): its derivative w (1 - w), of opposite signs
    p = torch.sigmoid(torch.where(idx == 1, z, -z))
    want = dw[:, 0].double() * p * (1 - p)
    got = d.double().gather(1, idx.long()[:, None])[:, 0]
    # an fp64 value rounded once to fp32; 1e-15 |dw| where 1 - s has cancelled
    assert torch.all((got - want).abs() <= 1e-7 * want.abs() + 1e-14 * dw[:, 0].abs())
    assert torch.all((d.double().sum(1)).abs() <= 2e-7 * want.abs() + 1e-14 * dw[:, 0].abs())
