"""The balance losses without a GPU: refusals, closed forms of the reference
and its gradient against differences."""
import numpy as np
import pytest
import torch

import balance_ref as ref
from mxfp4_weight_mixture_02_amd import BalanceLoss, moe_balance, moe_balance_backward, ops

FAKE = 0x10000   # never dereferenced: every call below returns from host checks
BIG = 1 << 60


def test_reference_closed_forms():
    """Even choices and probabilities: 1; all on one expert: E; a sequence
    alone counts as much as a longer one."""
    E = 4
    x = np.zeros((4, E))
    even = np.arange(4)[:, None]
    losses, counts, prob, n = ref.balance(x, even, "softmax")
    assert losses[0] == 1 and losses[1] == np.log(4) ** 2 and counts.tolist() == [[1] * 4] and n.tolist() == [4]
    hot = np.full((4, E), -200.0)
    hot[:, 1] = 0
    losses, _, _, _ = ref.balance(hot, np.ones((4, 1), int), "sigmoid")
    assert abs(losses[0] - 4) < 1e-12
    both = np.concatenate((hot, np.zeros((4, E))))
    idx = np.concatenate((np.ones((4, 1), int), even))
    losses, _, _, _ = ref.balance(both, idx, "softmax", offsets=[0, 4, 8])
    assert abs(losses[0] - 2.5) < 1e-12
    assert ref.balance(both, idx, "softmax", mask=np.zeros(8, bool))[0].tolist() == [0, 0]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_reference_gradient_against_differences(score):
    r = np.random.default_rng(0)
    x, idx = r.normal(size=(6, 5)) * 2, r.integers(0, 5, size=(6, 2))
    mask, offsets, dl = np.array([1, 1, 0, 1, 1, 1], bool), [0, 2, 2, 5], np.array([0.7, 0.3])
    g = ref.gradient(x, idx, score, dl, mask, offsets)
    assert not g[2].any() and not g[5].any()   # masked; behind the last sequence
    h = 1e-6   # off by h^2 of a third derivative and 1e-16 / h of the loss (below 10)
    for t in range(6):
        for e in range(5):
            d = np.zeros_like(x)
            d[t, e] = h
            num = (ref.balance(x + d, idx, score, mask, offsets)[0] - ref.balance(x - d, idx, score, mask, offsets)[0]) @ dl
            assert abs(num / (2 * h) - g[t, e]) < 1e-8


def _refused(code, rc):
    assert rc == code and ops.lib().mxfp4_last_error()


BAD = [(dict(T=0), -1), (dict(E=0), -1), (dict(k=0), -1), (dict(S=0), -1), (dict(S=65537), -2), (dict(E=257), -2),
       (dict(k=9), -2), (dict(E=3, k=4), -2), (dict(T=1 << 26), -2), (dict(score=2), -1), (dict(logits=None), -1),
       (dict(counts=None), -1), (dict(tokens=None), -1), (dict(S=2, off=None), -1), (dict(logits=FAKE + 2), -1),
       (dict(off=FAKE + 2), -1), (dict(counts=FAKE + 1), -1)]


@pytest.mark.parametrize("kw,code", BAD + [
    (dict(idx=None), -1), (dict(losses=None), -1), (dict(prob=None), -1), (dict(idx=FAKE + 2), -1), (dict(ws=None), -3),
    (dict(n=16), -3), (dict(ws=FAKE + 8), -1)])
def test_forward_refuses(kw, code):
    d = dict(score=0, T=300, E=8, k=4, S=1, logits=FAKE, idx=FAKE, mask=FAKE, off=FAKE, losses=FAKE, counts=FAKE,
             prob=FAKE, tokens=FAKE, ws=FAKE, n=BIG)
    d.update(kw)
    _refused(code, ops.lib().mxmoe_balance(*d.values(), None))


@pytest.mark.parametrize("kw,code", BAD + [
    (dict(dl=None), -1), (dict(out=None), -1), (dict(dl=FAKE + 2), -1), (dict(add=FAKE + 1), -1), (dict(out=FAKE + 2), -1)])
def test_backward_refuses(kw, code):
    d = dict(score=0, T=300, E=8, k=4, S=1, logits=FAKE, mask=FAKE, off=FAKE, counts=FAKE, tokens=FAKE, dl=FAKE,
             add=FAKE, out=FAKE)
    d.update(kw)
    _refused(code, ops.lib().mxmoe_balance_backward(*d.values(), None))


def test_workspace_query():
    f = ops.lib().mxmoe_balance_workspace_bytes
    assert 0 < f(1, 8, 2, 1) <= 256 < f(5000, 8, 2, 1) and f(100, 8, 2, 65536) > 65536 * 16
    for sizes in [(0, 8, 2, 1), (4, 300, 2, 1), (4, 8, 9, 1), (4, 8, 2, 0), (4, 8, 2, 65537)]:
        assert f(*sizes) == 0


def test_binding_refuses():
    x, idx, off = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.tensor([0, 4], dtype=torch.int32)
    b = BalanceLoss(None, torch.zeros(1, 8, dtype=torch.int32), None, torch.zeros(1, dtype=torch.int32), k=2)
    two = torch.zeros(2)
    for match, call in [
            (r"\[T, E\]", lambda: moe_balance(x[0], idx)),
            ("logits", lambda: moe_balance(x.double(), idx)),
            (r"\[T, k\]", lambda: moe_balance(x, idx[0])),
            ("topk_idx", lambda: moe_balance(x, idx.long())),
            ("topk_idx", lambda: moe_balance(x, idx[:3])),
            ("score", lambda: moe_balance(x, idx, score="relu")),
            ("mask", lambda: moe_balance(x, idx, mask=torch.ones(4))),
            ("mask", lambda: moe_balance(x, idx, mask=torch.ones(3, dtype=torch.bool))),
            ("offsets", lambda: moe_balance(x, idx, offsets=off[:1])),
            ("offsets", lambda: moe_balance(x, idx, offsets=off.long())),
            ("CUDA tensor", lambda: moe_balance(x, idx)),
            ("saved.counts", lambda: moe_balance_backward(x[:, :7].contiguous(), b, two)),
            ("dlosses", lambda: moe_balance_backward(x, b, two[:1])),
            ("add", lambda: moe_balance_backward(x, b, two, add=x[:3])),
            ("CUDA tensor", lambda: moe_balance_backward(x, b, two))]:
        with pytest.raises(ValueError, match=match):
            call()
