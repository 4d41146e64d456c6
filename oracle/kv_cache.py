"""The 8-bit cache of keys and values and the attention over it, float64. Test infrastructure.

A page holds `page` tokens of one sequence, [kv_heads, page, d] e4m3 values ("codes" as the numbers they stand for)
with a scale for each head; a value is code * scale. Writing: the smallest power of two s with |x| <= 448 s over the
new finite values, at least 2^-100; a part-filled page keeps the larger of its scale, rounded up to a power of two, and s,
and its codes are rounded again if that is larger than its scale. Codes are x / scale rounded to nearest, ties to
even; infinities and NaN become NaN, as do the codes of a part-filled page whose scale is not in (0, 2^120].
"""
import math

import numpy as np

from .attn_varlen import attn_varlen_fwd

E4M3 = np.array([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)][:127])


def e4m3_round(x):
    """Nearest e4m3 value (ties to the even code, beyond 448: 448); NaN for infinities and NaN."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(np.where(np.isfinite(x), x, 0.0)), 448.0)
    hi = np.searchsorted(E4M3, a)
    lo = np.maximum(hi - 1, 0)
    up, down = E4M3[hi] - a, a - E4M3[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return np.where(np.isfinite(x), np.copysign(E4M3[code], x), np.nan)


def page_scale(x):
    """The power of two that the finite values of x need."""
    a = np.abs(x[np.isfinite(x)])
    most = float(a.max()) if a.size else 0.0
    e = -100
    while most > math.ldexp(448.0, e):
        e += 1
    return math.ldexp(1.0, e)


def kv_cache_write(x, codes, scales, table, cu, start, page):
    """x [T, kv_heads, d] into codes [pages, kv_heads, page, d] and scales [pages, kv_heads], in place (float64)."""
    for i in range(len(cu) - 1):
        at, left, row = int(start[i]), int(cu[i + 1] - cu[i]), int(cu[i])
        while left > 0:
            pg, a = int(table[i][at // page]), at % page
            b = min(page, a + left)
            for h in range(x.shape[1]):
                new = np.asarray(x[row:row + b - a, h], dtype=np.float64)
                s = page_scale(new)
                if a > 0:
                    old = float(scales[pg, h])
                    if 0.0 < old <= 2.0 ** 120:
                        s = max(s, 2.0 ** math.ceil(math.log2(old)))
                        if s != old:
                            codes[pg, h, :a] = e4m3_round(codes[pg, h, :a] * (old / s))
                    else:
                        codes[pg, h, :a] = np.nan
                codes[pg, h, a:b] = e4m3_round(new / s)
                scales[pg, h] = s
            at, left, row = at + b - a, left - (b - a), row + b - a


def kv_cache_rows(codes, scales, pages, page, first, count):
    """Positions first .. first + count - 1 of a sequence with these pages: [count, kv_heads, d]."""
    out = np.zeros((count,) + (codes.shape[1], codes.shape[3]))
    for k in range(count):
        pg, slot = int(pages[(first + k) // page]), (first + k) % page
        out[k] = codes[pg, :, slot] * scales[pg][:, None]
    return out


def attn_cache_fwd(Q, kc, vc, ks, vs, table, cu_q, lens, page, causal, scale):
    """O [Tq, heads, d], LSE [heads, Tq]."""
    k, v = ([kv_cache_rows(c, s, table[i], page, 0, int(lens[i])) for i in range(len(lens))]
            for c, s in ((kc, ks), (vc, vs)))
    cu_k = np.concatenate([[0], np.cumsum(lens)]).astype(int)
    return attn_varlen_fwd(Q, np.concatenate(k), np.concatenate(v), cu_q, cu_k, causal, scale)
