"""The attention over the 8-bit cache where values are near the largest of their type: O is a mean of values, so it is as large
as they are at most.

Tolerance per element of O, from the row's own tokens: half a bf16 step (2^-8), the probabilities' rounding to halves (2^-11 of
each) and the scores' error as in test_gpu_attn_cache, relative to A = sum P |v|; and a half's least step, 2^-25 where the
largest P * scale of the row is 2^7 at least, for each token: 2^-32 of that product times a code (448 at most)."""
import numpy as np
import pytest
import torch

import oracle
from cache_util import f64
from gpu_util import mp
from test_gpu_attn_cache import _make, _run

pytestmark = pytest.mark.gpu


def _check(got, inp, new, lens, causal=True, scale=None):
    Q, codes, scales, table = inp
    O, LSE = f64(got[0]), f64(got[1])
    heads, d, kv, page = Q.shape[1], Q.shape[2], codes.shape[2], codes.shape[3]
    scale = d ** -0.5 if scale is None else scale
    q, row = f64(Q), 0
    for i, (nq, nk) in enumerate(zip(new, lens)):
        pages = table[i].tolist()
        k, v = (oracle.kv_cache_rows(f64(codes[:, j]), f64(scales[:, j]), pages, page, 0, nk) for j in (0, 1))
        vs = np.stack([f64(scales[pages[t // page], 1]) for t in range(nk)])  # [nk, kv]
        for n in range(nq):
            sees = nk - nq + n + 1 if causal else nk
            at = q[row + n:row + n + 1]
            wo, wl = oracle.attn_varlen_fwd(at, k[:sees], v[:sees], [0, 1], [0, sees], False, scale)
            wa, _ = oracle.attn_varlen_fwd(at, k[:sees], np.abs(v[:sees]), [0, 1], [0, sees], False, scale)
            kk = np.repeat(k[:sees], heads // kv, axis=1)
            z = scale * np.einsum("hd,khd->hk", at[0], kk)
            most = scale * np.einsum("hd,khd->hk", np.abs(at[0]), np.abs(kk)).max(-1)
            es = 2.0 ** -20 * most + 2.0 ** -20
            weight = (np.exp(z - wl) * np.repeat(vs[:sees], heads // kv, axis=1).T).max(-1)  # [heads]
            tol = (2.0 ** -8 * np.abs(wo[0]) + (2.0 ** -11 + 2 * es[:, None]) * wa[0]
                   + 2.0 ** -32 * 448 * sees * weight[:, None])
            err = np.abs(O[row + n] - wo[0]) - tol
            assert np.all(err <= 0), (i, n, float(np.max(np.abs(O[row + n] - wo[0]) / tol)))
            le = np.abs(LSE[:, row + n] - wl[:, 0]) - (es + 2.0 ** -21 * (1 + np.abs(wl[:, 0])))
            assert np.all(le <= 0), (i, n, float(le.max()))
        row += nq


@pytest.mark.parametrize("new,lens,heads,kv,d,page", [
    ([1], [1], 2, 1, 64, 16),            # one key: finished from registers
    ([2, 1], [300, 40], 4, 2, 96, 32),   # a CTA's records
    ([1], [20000], 8, 1, 64, 64),        # parts of many CTAs
    ([3], [9000], 16, 2, 128, 128),      # the same, rows of two tiles' width
])
@pytest.mark.parametrize("e", [100, 113, 118])
def test_values_near_the_largest(new, lens, heads, kv, d, page, e):
    Q, codes, scales, table = _make(new, lens, heads, kv, d, page, 26000 + d, spread=1)
    scales[:, 1] *= 2.0 ** e * 64
    v = codes.float()[:, 1] * scales[:, 1, :, None, None]
    assert not torch.isinf(v).any()
    inp = Q, codes, scales, table
    _check(_run(*inp, new, lens), inp, new, lens)
