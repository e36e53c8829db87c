"""8-bit block formats and products in float64 numpy (test helper)."""
import numpy as np

from oracle.mxfp8 import e4m3_decode, e4m3_round


def bf16(x):
    """Nearest bf16 values of float32 x, ties to even, as float32."""
    b = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    return ((b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)


def exponents(amax):
    """The smallest e with amax <= 448 * 2^e, at least -127."""
    e = np.full(amax.shape, -127, dtype=np.int64)
    nz = amax > 0
    g = np.floor(np.log2(amax[nz])).astype(np.int64) - 9
    for _ in range(3):
        g = np.where(np.ldexp(448.0, g) < amax[nz], g + 1, g)
    e[nz] = np.maximum(g, -127)
    return e


def quantize(x, block_rows, block):
    """(codes [rows, K rounded up to block], exponents [row blocks, K blocks])."""
    x = np.asarray(x, dtype=np.float64)
    rows, K = x.shape
    kb, rb = -(-K // block), -(-rows // block_rows)
    p = np.zeros((rb * block_rows, kb * block))
    p[:rows, :K] = x
    t = p.reshape(rb, block_rows, kb, block)
    ok = np.isfinite(t)
    e = exponents(np.where(ok, np.abs(t), 0).max(axis=(1, 3)))
    y = np.ldexp(np.where(ok, t, 0), -e[:, None, :, None])
    codes = np.where(ok, e4m3_round(y), 0x7F).reshape(p.shape)[:rows]
    nan = ~ok.reshape(p.shape)[:rows]
    return codes.astype(np.uint8), e, nan


def values(codes, e, block_rows, block):
    rows = codes.shape[0]
    f = np.repeat(np.repeat(e, block_rows, 0)[:rows], block, 1)
    return np.ldexp(e4m3_decode(codes), f)


def rounded(x, block_rows=1, block=128):
    """x on its blocks' E4M3 grids."""
    c, e, _ = quantize(x, block_rows, block)
    return values(c, e, block_rows, block)[:, :x.shape[1]]


def scale_bytes(e, block_rows, rows):
    """The library's scale layout: [K blocks, rows rounded up to 16 | row blocks]."""
    s = (e.T + 127).astype(np.uint8)
    if block_rows == 1:
        out = np.zeros((s.shape[0], -(-rows // 16) * 16), np.uint8)
        out[:, :rows] = s
        return out
    return s


def swiglu_codes(h, limit):
    """MXFP8 codes of h [R, 2I] kept on their values' sides of the clamp bounds,
    and the exponents [R, 2I / 32]."""
    codes, e, nan = quantize(h, 1, 32)
    v = values(codes, e, 1, 32)
    h = np.asarray(h, np.float64)
    up = np.arange(h.shape[1]) % 2 == 1
    with np.errstate(invalid="ignore"):
        d = (h > limit).astype(int) - (v > limit) + up * ((h < -limit).astype(int) - (v < -limit))
    return np.where(nan, codes, codes + d).astype(np.uint8), e


def swiglu(h, alpha, limit):
    g, u = np.minimum(h[:, 0::2], limit), np.clip(h[:, 1::2], -limit, limit)
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-alpha * g)) * (u + 1)


def swiglu_grad(h, da, alpha, limit):
    g, u = np.minimum(h[:, 0::2], limit), np.clip(h[:, 1::2], -limit, limit)
    with np.errstate(over="ignore"):
        s = 1 / (1 + np.exp(-alpha * g))
    out = np.empty_like(h)
    out[:, 0::2] = da * (u + 1) * s * (1 + alpha * g * (1 - s)) * (h[:, 0::2] <= limit)
    out[:, 1::2] = da * g * s * (np.abs(h[:, 1::2]) <= limit)
    return out
