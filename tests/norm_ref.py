"""The root-mean-square norm and its gradients in float64 numpy (test helper)."""
import numpy as np

from fp8_ref import bf16


def stream(x, r, f32):
    """x + r as it is stored: one fp32 addition, rounded to the tensors' type."""
    if r is None:
        return np.asarray(x, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        s = np.asarray(x, np.float32) + np.asarray(r, np.float32)
    return (s if f32 else bf16(s)).astype(np.float64)


def norm(s, w, eps):
    """(y, rstd) of the rows of s."""
    rstd = 1 / np.sqrt((s * s).mean(1) + eps)
    return s * rstd[:, None] * w, rstd


def backward(s, rstd, w, dy, ds=None):
    """(dx, dw, and the magnitudes that their sums pass through)."""
    xhat = s * rstd[:, None]
    g = dy * w
    dot, mag = (g * xhat).mean(1, keepdims=True), np.abs(g * xhat).mean(1, keepdims=True)
    dx = rstd[:, None] * (g - xhat * dot)
    size = rstd[:, None] * (np.abs(g) + np.abs(xhat) * mag)
    if ds is not None:
        dx, size = dx + ds, size + np.abs(ds)
    return dx, (dy * xhat).sum(0), size, np.abs(dy * xhat).sum(0)
