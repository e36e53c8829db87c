"""MXFP4 matrices in the products' layouts (test helper): the oracle's
quantizer, with rows padded and non-finite blocks marked."""
import numpy as np
import torch

from oracle import mxfp4


def quantize(x):
    """(codes [rows, K rounded up to 256, / 2], scales [rows, K rounded up to
    256, / 32]) of float32 x [rows, K]; scales past K are 0."""
    x = np.asarray(x, np.float32)
    rows, K = x.shape
    p = np.zeros((rows, -(-K // 256) * 256), np.float32)
    p[:, :K] = x
    bad = ~np.isfinite(p.reshape(rows, -1, 32)).all(2)
    codes, scales = mxfp4.quantize(np.where(np.repeat(bad, 32, 1), 0, p))
    return codes, np.where(bad, 255, scales).astype(np.uint8)


def ordered(scales):
    """Scales [rows, K blocks * 8] in the products' order, rows padded with 0."""
    rows, n = scales.shape
    p = np.zeros((-(-rows // 16) * 16, -(-n // 8) * 8), np.uint8)
    p[:rows, :n] = scales
    return p.reshape(p.shape[0], -1, 4, 2).transpose(1, 2, 0, 3)


def natural(q):
    """An Fp4Matrix's scales as [rows, K blocks * 8]."""
    s = q.scales.cpu().numpy()
    return s.transpose(2, 0, 1, 3).reshape(s.shape[2], -1)[:q.rows]


def values(q):
    """float64 [rows, K] that an Fp4Matrix stands for."""
    s = natural(q)[:, :-(-q.K // 32)]
    c = mxfp4.unpack_codes(q.codes.cpu().numpy())
    p = np.zeros((q.rows, s.shape[1] * 32), np.uint8)
    n = min(p.shape[1], c.shape[1])
    p[:, :n] = c[:, :n]
    with np.errstate(invalid="ignore"):
        return (mxfp4.e2m1_decode(p) * np.repeat(mxfp4.ue8m0_decode(s), 32, 1))[:, :q.K]


def whole(rows, K, g, device, span=2):
    """float32 [rows, K] of integers up to 3 times a power of two for each
    block of 32: MXFP4 holds them exactly."""
    v = torch.randint(-3, 4, (rows, K), generator=g, device=device).float()
    e = torch.randint(-span, span + 1, (rows, -(-K // 32)), generator=g, device=device).float().exp2()
    return v * e.repeat_interleave(32, 1)[:, :K]
