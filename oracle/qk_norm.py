"""Norm of queries and keys for each head with the rotation, forward and backward, float64. Test infrastructure.

n = x / sqrt(mean(x^2) + eps) over a head's elements, y = R(w * n): w = wq for the first q_heads heads, wk for the
others, R the rotation of ``rope``. Its gradients: g = R^-1 dy, dw = sum of g * n over tokens and heads,
dx = (w * g - n mean(w * g * n)) / sqrt(mean(x^2) + eps).
"""
import numpy as np

from .rope import rope


def _parts(x, wq, wk, q_heads, eps):
    x = np.asarray(x, dtype=np.float64)
    r = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    w = np.stack([np.asarray(wq if h < q_heads else wk, dtype=np.float64) for h in range(x.shape[1])])
    return x * r, r, w


def qk_norm_rope(x, wq, wk, pos, q_heads, sections, base, eps, interleaved=False, per_axis=False):
    n, _, w = _parts(x, wq, wk, q_heads, eps)
    return rope(n * w, pos, sections, base, interleaved, per_axis)


def qk_norm_rope_bwd(x, dy, wq, wk, pos, q_heads, sections, base, eps, interleaved=False, per_axis=False):
    """dict of dx, dwq, dwk."""
    n, r, w = _parts(x, wq, wk, q_heads, eps)
    g = rope(dy, pos, sections, base, interleaved, per_axis, inverse=True)
    dw = (g * n).sum(axis=0)
    dx = r * (w * g - n * np.mean(w * g * n, axis=-1, keepdims=True))
    return {"dx": dx, "dwq": dw[:q_heads].sum(axis=0), "dwk": dw[q_heads:].sum(axis=0)}
