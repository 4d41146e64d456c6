"""Rotary positions with several axes, float64. Test infrastructure.

A head's 2n rotated elements form n pairs (a, b): pair i at elements (i, i + n), or (2i, 2i + 1)
when interleaved. Axis k owns the k-th run of sections[k] pairs; pair i turns by
pos[axis(i)] * base^(-i / n), or base^(-j / sections[axis]) for the j-th pair of its axis
(``per_axis``). The remaining elements pass through. The rotation is orthogonal: its gradient is
the rotation back.
"""
import numpy as np


def rope_angles(pos, sections, base, per_axis):
    """[T, n] angles in radians."""
    pos = np.asarray(pos, dtype=np.float64)
    n = int(sum(sections))
    cols = []
    for axis, size in enumerate(sections):
        for j in range(size):
            e = j / size if per_axis else len(cols) / n
            cols.append(pos[axis] * float(base) ** -e)
    return np.stack(cols, axis=1) if cols else np.zeros((pos.shape[1], 0))


def rope(x, pos, sections, base, interleaved=False, per_axis=False, inverse=False):
    """x [T, heads, d] rotated."""
    x = np.asarray(x, dtype=np.float64)
    n = int(sum(sections))
    ang = rope_angles(pos, sections, base, per_axis)
    if inverse:
        ang = -ang
    c, s = np.cos(ang)[:, None, :], np.sin(ang)[:, None, :]
    ia = np.arange(n) * 2 if interleaved else np.arange(n)
    ib = ia + 1 if interleaved else ia + n
    y = x.copy()
    y[..., ia] = x[..., ia] * c - x[..., ib] * s
    y[..., ib] = x[..., ib] * c + x[..., ia] * s
    return y
