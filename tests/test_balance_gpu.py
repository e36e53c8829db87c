"""The balance losses on the GPU against float64: sizes, ragged and empty
sequences, masks, extreme logits, gradients, graphs."""
import numpy as np
import pytest
import torch

import balance_ref as ref
from gpu_helpers import to_f64
from mxfp4_weight_mixture_02_amd import (RouteOptions, moe_balance, moe_balance_backward, moe_route, moe_route_backward,
                                         ops)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
# A probability: an exponential's argument is rounded at |x - m| <= 30 (2^-20
# of the value), the exponential, the sum of at most 256 and the quotient add
# less than 32 roundings of 2^-24; its mean sums at most 32 tokens a row of
# lanes (1024 tokens a workgroup, 32 at a time) and 32 rows in fp32.
P = 2.0 ** -20 + 128 * 2.0 ** -24
SIZES = [(1, 1, 1), (1, 256, 8), (7, 2, 1), (64, 32, 4), (255, 100, 6), (256, 7, 3), (257, 64, 8), (1000, 65, 2),
         (5000, 128, 4), (3001, 256, 8), (40000, 30, 2)]


def _draw(T, E, k, seed=0, std=1.5, shift=0):
    r = np.random.default_rng(seed)
    x = (r.normal(size=(T, E)) * std).astype(np.float32)
    idx = np.argsort(-x, axis=1)[:, :k].astype(np.int32)
    flat = torch.empty(T * E + shift, device=DEV)
    d = flat[shift:].view(T, E)
    d.copy_(torch.from_numpy(x))
    return x, idx, d, torch.from_numpy(idx).to(DEV)


def _check(b, x, idx, score, mask=None, offsets=None):
    losses, counts, prob, n = ref.balance(x, idx, score, mask, offsets)
    assert np.array_equal(b.counts.cpu().numpy(), counts) and np.array_equal(b.tokens.cpu().numpy(), n)
    # below 2^-126 a probability's parts may have underflowed
    assert np.all(np.abs(to_f64(b.prob) - prob) <= prob * P + 2.0 ** -126)
    got = to_f64(b.losses)
    assert abs(got[0] - losses[0]) <= losses[0] * (P + 2.0 ** -23)
    # lse: m + log(sum), 2^-22 of |m| + log 256; its square doubles that
    big = np.abs(x[np.isfinite(x)]).max() + np.log(256) if np.isfinite(x).any() else 0
    assert abs(got[1] - losses[1]) <= big * big * (2.0 ** -21 + 128 * 2.0 ** -24)


def _check_grad(d, x, idx, score, dl, mask=None, offsets=None, add=None):
    g = ref.gradient(x, idx, score, dl, mask, offsets)
    p, soft, lse, rest = ref.probabilities(x, score)
    _, counts, _, n = ref.balance(x, idx, score, mask, offsets)
    size = np.zeros_like(g)
    for t, c, m in zip(ref.tokens_of(x.shape[0], mask, offsets), counts, n):
        if m:
            f = np.abs(dl[0]) * x.shape[1] * c / (idx.shape[1] * m * m * (n > 0).sum())
            big = np.abs(x[t]).max() + np.log(256)
            size[t] = p[t] * (f + (f * p[t]).sum(1, keepdims=True)) + 2 * abs(dl[1]) / n.sum() * big * soft[t]
    want = g if add is None else g + add
    # twice a probability's error, and the last roundings
    tol = size * (2 * P + 2.0 ** -21) + np.abs(want) * 2.0 ** -23 + 2.0 ** -126
    assert np.all(np.abs(to_f64(d) - want) <= tol)


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("score,shift", [("softmax", 0), ("sigmoid", 0), ("sigmoid", 1)])
def test_one_sequence(T, E, k, score, shift):
    print("balance", T, E, k, score, shift, flush=True)
    x, idx, d, di = _draw(T, E, k, shift=shift)
    mask = np.random.default_rng(1).random(T) < 0.8
    dl = torch.tensor([0.01, 0.001], device=DEV)
    for m in (None, mask):
        dm = None if m is None else torch.from_numpy(m).to(DEV)
        b = moe_balance(d, di, score=score, mask=dm)
        _check(b, x, idx, score, m)
        _check_grad(moe_balance_backward(d, b, dl), x, idx, score, to_f64(dl), m)
        again = moe_balance(d, di, score=score, mask=dm)
        assert torch.equal(again.losses, b.losses) and torch.equal(again.prob, b.prob)


# ragged, empty, single-token sequences; ones that end inside and at the end of
# a workgroup's tokens; tokens before the first and behind the last
CUTS = {
    "whole": lambda T: [0, T], "inner": lambda T: [T // 4, T // 2], "empty": lambda T: [T // 2, T // 2],
    "none": lambda T: [0, 0, 0, 0], "ragged": lambda T: sorted([0, T // 3, T // 3, T // 3 + 1, T // 2, T - 1, T]),
    "blocks": lambda T: [min(T, 128 * i) for i in range(T // 128 + 2)],
    "ones": lambda T: list(range(min(T, 200) + 1)), "clamped": lambda T: [-5, 2, T + 10, T + 20],
    "many": lambda T: sorted(np.random.default_rng(3).integers(0, T + 1, size=400).tolist())}


@pytest.mark.parametrize("T,E,k", [(5, 9, 2), (256, 16, 4), (300, 70, 8), (3000, 256, 8), (9000, 32, 4)])
@pytest.mark.parametrize("cuts", sorted(CUTS))
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_sequences(T, E, k, cuts, score):
    print("balance", T, E, k, cuts, score, flush=True)
    x, idx, d, di = _draw(T, E, k, seed=2)
    off = CUTS[cuts](T)
    mask = np.random.default_rng(4).random(T) < 0.7
    add = np.random.default_rng(5).normal(size=(T, E)).astype(np.float32)
    doff = torch.tensor(off, dtype=torch.int32, device=DEV)
    dm = torch.from_numpy(mask).to(DEV)
    b = moe_balance(d, di, score=score, mask=dm, offsets=doff)
    _check(b, x, idx, score, mask, off)
    dl = torch.tensor([1.0, -0.5], device=DEV)
    got = moe_balance_backward(d, b, dl, add=torch.from_numpy(add).to(DEV))
    _check_grad(got, x, idx, score, to_f64(dl), mask, off, add)
    alone = moe_balance_backward(d, b, dl)
    _check_grad(alone, x, idx, score, to_f64(dl), mask, off)
    live = np.zeros(T, bool)
    for t in ref.tokens_of(T, mask, off):
        live[t] = True
    left = torch.from_numpy(~live).to(DEV)
    assert torch.all(alone[left] == 0) and torch.equal(got[left].cpu(), torch.from_numpy(add)[~live])


@pytest.mark.parametrize("T,E", [(9, 12), (300, 33)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_extreme_logits(T, E, score):
    """Experts shut with -inf and with the lowest finite value, a token with
    nothing open, logits far apart and all far below zero."""
    x, idx, _, di = _draw(T, E, 2, seed=6)
    x[0, :] = -np.inf
    x[1, 1:] = -np.inf
    x[2, ::2] = np.finfo(np.float32).min
    x[3] = -150 - np.arange(E)
    x[4, 3] = 3e4
    x[5] += 80
    idx[6] = [-1, E]
    d, di = torch.from_numpy(x).to(DEV), torch.from_numpy(idx).to(DEV)
    b = moe_balance(d, di, score=score)
    _, counts, prob, n = ref.balance(x, idx, score)
    assert np.array_equal(b.counts.cpu().numpy(), counts) and b.counts.sum() == 2 * T - 2
    # an argument of |x - m| <= 300 rounds by 2^-16 of the value
    assert np.all(np.abs(to_f64(b.prob) - prob) <= prob * (2.0 ** -16 + P) + 2.0 ** -126)
    assert torch.isfinite(b.losses).all()
    dl = torch.tensor([1.0, 0.0], device=DEV)
    g, w = to_f64(moe_balance_backward(d, b, dl)), ref.gradient(x, idx, score, [1.0, 0.0])
    assert np.all(np.isfinite(g)) and not g[0].any()
    top = E * counts.max() / (2 * T * T)
    assert np.all(np.abs(g - w) <= 2 * top * (2.0 ** -16 + P))


@pytest.mark.parametrize("T", [20, 700])
def test_a_nan_token_keeps_to_itself(T):
    x, idx, _, _ = _draw(T, 16, 2, seed=7)
    x[3, 5] = np.nan
    d, di = torch.from_numpy(x).to(DEV), torch.from_numpy(idx).to(DEV)
    mask = torch.ones(T, dtype=torch.bool, device=DEV)
    b = moe_balance(d, di, mask=mask)
    g = moe_balance_backward(d, b, torch.ones(2, device=DEV))
    assert torch.isnan(b.losses).all() and torch.isnan(g[3]).all() and torch.isfinite(g[4:]).all()
    # masked, it is not read into anything
    mask[3] = False
    b = moe_balance(d, di, mask=mask)
    g = moe_balance_backward(d, b, torch.ones(2, device=DEV))
    assert torch.isfinite(b.losses).all() and torch.isfinite(g).all() and not g[3].any()


def test_large_batch_and_many_sequences():
    """More parts than one workgroup sums at once: 2^20 tokens of one sequence,
    then 65536 sequences of 1 to 31 tokens."""
    T, E = 1 << 20, 16
    g = torch.Generator(device=DEV).manual_seed(8)
    x = torch.randn(T, E, generator=g, device=DEV)
    idx = x.sort(dim=1, descending=True).indices[:, :2].to(torch.int32).contiguous()
    b = moe_balance(x, idx)
    assert torch.equal(b.counts[0], torch.bincount(idx.flatten().long(), minlength=E).int())
    want = torch.softmax(x.double(), 1).mean(0)
    assert torch.all((b.prob[0].double() - want).abs() <= want * P)
    off = torch.linspace(0, T, 65537, device=DEV).to(torch.int32)
    b = moe_balance(x, idx, offsets=off)
    n = (off[1:] - off[:-1]).long()
    assert torch.equal(b.tokens, n.int())
    seg = torch.repeat_interleave(torch.arange(65536, device=DEV), n)
    prob = torch.zeros(65536, E, dtype=torch.float64, device=DEV).index_add_(0, seg, torch.softmax(x.double(), 1))
    assert torch.all((b.prob.double() - prob / n[:, None]).abs() <= prob / n[:, None] * P + 1e-30)
    hot = torch.zeros(65536 * E, dtype=torch.int32, device=DEV)
    hot.index_add_(0, (seg[:, None] * E + idx.long()).flatten(), torch.ones(2 * T, dtype=torch.int32, device=DEV))
    assert torch.equal(b.counts.flatten(), hot)
    f = b.counts.double() / (2 * n[:, None])
    loss = (E * f * prob / n[:, None]).sum(1).mean()
    assert abs(float(b.losses[0]) - float(loss)) <= float(loss) * (P + 2.0 ** -23)
    d = moe_balance_backward(x, b, torch.tensor([1.0, 0.0], device=DEV))
    p = torch.softmax(x.double(), 1)
    c = (E * f / n[:, None] / 65536)[seg]
    w = p * (c - (c * p).sum(1, keepdim=True))
    assert torch.all((d.double() - w).abs() <= p * (c + (c * p).sum(1, keepdim=True)) * (2 * P + 2.0 ** -21) + 1e-30)


def test_dlogits_over_add():
    x, idx, d, di = _draw(50, 10, 2)
    b = moe_balance(d, di)
    dl, add = torch.ones(2, device=DEV), torch.randn(50, 10, device=DEV)
    want = moe_balance_backward(d, b, dl, add=add)
    p = lambda t: t.data_ptr()  # noqa: E731
    assert ops.lib().mxmoe_balance_backward(0, 50, 10, 2, 1, p(d), None, None, p(b.counts), p(b.tokens), p(dl), p(add),
                                            p(add), torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(add, want)


@pytest.mark.parametrize("T", [20, 1500])
def test_router_step_captured(T):
    """Routing, its losses and their gradients: two graphs replayed in turn with
    eager steps between give the eager bits."""
    E, k, o = 24, 3, RouteOptions(score="sigmoid")
    g = torch.Generator(device=DEV).manual_seed(9)
    xs = [torch.randn(T, E, generator=g, device=DEV) for _ in range(3)]
    off = torch.tensor([0, T // 3, T - 2], dtype=torch.int32, device=DEV)
    dl, dw = torch.tensor([0.01, 0.001], device=DEV), torch.randn(T, k, generator=g, device=DEV)

    def step(x):
        r = moe_route(x, k, o)
        out = []
        for offsets in (None, off):
            b = moe_balance(x, r.topk_idx, score="sigmoid", offsets=offsets)
            out += [b.losses, b.counts, b.prob, b.tokens,
                    moe_balance_backward(x, b, dl, add=moe_route_backward(x, r.topk_idx, dw, o))]
        return out

    want = [step(x) for x in xs]
    assert torch.equal(want[0][1][0], torch.diff(moe_route(xs[0], k, o).expert_offsets))
    hold = [xs[0].clone(), xs[1].clone()]
    graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for gr, h in zip(graphs, hold):
        with torch.cuda.graph(gr):
            outs.append(step(h))
    for i in range(4):
        for h, j in zip(hold, (i % 3, (i + 1) % 3)):
            h.copy_(xs[j])
        step(xs[2])
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for o_, j in zip(outs, (i % 3, (i + 1) % 3)):
            assert all(torch.equal(a, b) for a, b in zip(o_, want[j]))
