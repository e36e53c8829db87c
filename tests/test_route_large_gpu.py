"""Routing of large batches: workgroups whose rows take several turns of the
scatter (more than 8192 tokens with k = 8), waves that take several tokens,
and more histograms than the prefix sum has threads (above 65536 tokens).

Integers are equal; a weight is an fp64 value rounded once to fp32 (1e-7)."""
import numpy as np
import pytest
import torch

import route_grad_ref as ref
from mxfp4_weight_mixture_02_amd import RouteOptions, moe_route

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("T,E,k,o", [
    (9001, 32, 8, RouteOptions()),
    (16385, 256, 8, RouteOptions(score="sigmoid", groups=8, top_groups=4, scale=2.5)),
    (16385, 250, 8, RouteOptions()),          # E % 4: one token a wave
    (40003, 128, 8, RouteOptions()),
    (40003, 126, 7, RouteOptions(score="sigmoid", groups=9, top_groups=2)),
    (65537, 16, 8, RouteOptions(renorm=False)),
    (70001, 256, 8, RouteOptions(score="sigmoid")),
    (70001, 254, 8, RouteOptions(score="sigmoid", renorm=False)),
    (140001, 24, 3, RouteOptions())])
@pytest.mark.parametrize("skewed", [False, True])
def test_plan(T, E, k, o, skewed):
    """Logits in steps of 1/16, so that many are equal and the others differ by
    far more than an exponential's error; skewed: most tokens take the same
    few experts, so that a chunk's rows crowd into one place."""
    print("route", T, E, k, o, skewed, flush=True)
    r = np.random.default_rng(T + E)
    x = (np.round(r.normal(size=(T, E)) * 24) / 16).astype(np.float32)
    if skewed:
        x[: T * 2 // 3, E // 3: E // 3 + 3] += 6
        x[T * 5 // 6:, 0] += 9
    bias = (r.integers(-4, 5, size=E) / 32).astype(np.float32) if E % 8 == 0 else None
    got = moe_route(torch.from_numpy(x).to(DEV), k, o, bias=None if bias is None else torch.from_numpy(bias).to(DEV))
    idx, w, off, rows = ref.route(x, k, o, bias)
    assert np.array_equal(got.topk_idx.cpu().numpy(), idx)
    assert np.array_equal(got.expert_offsets.cpu().numpy(), off)
    assert np.array_equal(got.sorted_rows.cpu().numpy(), rows)
    np.testing.assert_allclose(got.topk_w.cpu().numpy(), w, rtol=1e-7)
