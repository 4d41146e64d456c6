"""The attention over the 8-bit cache where values' scales are large or far apart: O is a mean of values, so it is as large as they
are at most, and a row's result goes by the tokens that have weight in it.

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


def _check(got, inp, new, lens, causal=True, scale=None, only=None):
    Q, codes, scales, table = inp
    O, LSE = f64(got[0]), f64(got[1])
    heads, d, kv, page = Q.shape[1], Q.shape[2], codes.shape[2], codes.shape[3]
    scale = d ** -0.5 if scale is None else scale
    q, row = f64(Q), 0
    for i, (nq, nk) in enumerate(zip(new, lens)):
        if only is not None and i not in only:
            row += nq
            continue
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


def _far(inp, i, j, by, page):
    """The value scale of the page that holds token j of sequence i, times 2^by."""
    inp[2][int(inp[3][i, j // page]), 1] *= 2.0 ** by


@pytest.mark.parametrize("by", [21, 40, 90])
def test_pages_that_a_causal_row_does_not_see(by):
    # the last two tokens of each sequence have a page of their own, which the first query of three does not see
    new, lens, page = [3, 3], [16 * 5 + 2, 16 * 700 + 2], 16
    inp = _make(new, lens, 4, 2, 64, page, 26100, spread=1)
    for i, n in enumerate(lens):
        _far(inp, i, n - 1, by, page)
    _check(_run(*inp, new, lens), inp, new, lens)


@pytest.mark.parametrize("by", [40, 90])
@pytest.mark.parametrize("where", [0, 20, -1])
@pytest.mark.parametrize("d,page", [(64, 16), (96, 32), (128, 64)])
def test_pages_without_weight(by, where, d, page):
    # one page's keys turn away from the queries (scores some 200 below the others'), its values are far larger; a warp walks
    # ten tiles and more on end
    heads, kv, n = 16, 8, 2000
    new, lens = [1] * 24, [n] * 24
    Q, codes, scales, table = inp = _make(new, lens, heads, kv, d, page, 26200, spread=0)
    Q[:] = Q.abs() + 0.5
    scales[:, 0] *= 2.0 ** -3
    for i in range(len(new)):
        at = where * page if where >= 0 else n - 1
        pg = int(table[i, at // page])
        away = -(codes[pg, 0].float().nan_to_num(0).abs() + 64).clamp(max=448)
        codes[pg, 0] = away.to(codes.dtype)
        scales[pg, 0] = 2.0
        _far(inp, i, at, by, page)
    _check(_run(*inp, new, lens, scale=0.01), inp, new, lens, scale=0.01, only=(0, 11, 23))


def test_zero_and_tiny_scales_beside_ordinary_ones():
    # pages of zeros at the least scale that a write leaves, one with the scale zero, and scores that rise towards them
    new, lens, page = [1, 2], [700, 90], 16
    Q, codes, scales, table = inp = _make(new, lens, 4, 2, 64, page, 26300, spread=8)
    for i, n in enumerate(lens):
        for t in range(0, n, 3 * page):
            pg = int(table[i, t // page])
            codes[pg, 1] = 0
            scales[pg, 1] = 2.0 ** -100 if t % (2 * page) else 0.0
            scales[pg, 0] *= 8
    _check(_run(*inp, new, lens), inp, new, lens)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_scale_that_is_no_number_reaches_the_rows_that_see_it(bad):
    new, lens, page = [3, 1], [16 * 12 + 1, 90], 16
    Q, codes, scales, table = _make(new, lens, 4, 2, 64, page, 26400)
    clean = _run(Q, codes, scales, table, new, lens)
    scales[int(table[0, 12]), 1, 1] = bad  # the last query alone sees that page, heads 2 and 3 read it
    O, LSE = _run(Q, codes, scales, table, new, lens)
    hit = torch.zeros(4, 4, dtype=torch.bool)
    hit[2, 2:] = True
    assert torch.isnan(O[hit]).all() and torch.isnan(LSE.t()[hit]).all()
    assert torch.equal(O[~hit], clean[0][~hit]) and torch.equal(LSE.t()[~hit], clean[1].t()[~hit])


@pytest.mark.parametrize("by", [30, 100, 125, 150, 190, 215])
@pytest.mark.parametrize("first", [0, 1, 2])
@pytest.mark.parametrize("page", [16, 64])
def test_small_probabilities_of_large_values(by, first, page):
    # every third page's tokens have 2^-by of the others' probability and 2^by times their values: both count alike
    heads, kv, d = 16, 8, 64
    new, lens = [1] * 12 + [2], [600] * 12 + [90]
    Q, codes, scales, table = inp = _make(new, lens, heads, kv, d, page, 26500, spread=0)
    Q[:] = 0
    Q[..., 5] = 1.0
    scales[:, 0] = 1.0
    for i, n in enumerate(lens):
        for k in range(-(-n // page)):
            pg, far = int(table[i, k]), k % 3 == first
            codes[pg, 0, :, :, 5] = -448.0 if far else 0.0
            scales[pg, 1] = 2.0 ** (110 - (0 if far else by))
    how = dict(scale=by * float(np.log(2.0)) / 448)
    _check(_run(*inp, new, lens, **how), inp, new, lens, only=(0, 11, 12), **how)


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("top", [1e3, 1e5, 1.05e6, 4.2e6, 1e8, 1e9, 1e12, 1e20, 1e37])
@pytest.mark.parametrize("n,at", [(90, 3), (90, 88), (3000, 1501)])
def test_large_scores_give_the_value_of_the_largest(sign, top, n, at):
    # one key's score is 7 % or more above all others', so that its value is the result
    heads, kv, d, page = 4, 2, 64, 32
    Q, codes, scales, table = _make([1, 1], [n, 40], heads, kv, d, page, 26600, spread=0)
    g = torch.Generator().manual_seed(1)
    Q[:] = 0
    Q[0, :, 7] = float(np.float32(top))  # bf16 rounds it, for all keys alike
    scales[:, 0] = 1.0 / 448
    for k in range(-(-n // page)):
        low = torch.randint(1, 13, (kv, page), generator=g).float() * 32  # 32 .. 384
        codes[int(table[0, k]), 0, :, :, 7] = low if sign > 0 else -448.0
    codes[int(table[0, at // page]), 0, :, at % page, 7] = 448.0 if sign > 0 else -416.0
    O, LSE = _run(Q, codes, scales, table, [1, 1], [n, 40], scale=1.0)
    pg = int(table[0, at // page])
    want = codes[pg, 1, :, at % page].float() * scales[pg, 1][:, None]
    assert torch.equal(O[0].float(), want.repeat_interleave(2, 0))
    s = float(Q[0, 0, 7]) * (1.0 if sign > 0 else -416.0 / 448)
    assert torch.all((LSE[:, 0].double() - s).abs() <= 2.0 ** -19 * abs(s))


def test_log_sum_exp_of_few_keys():
    """Scores of one product each, up to 4: what is left are roundings. A score's (two of 2^-24 of it, 1.4e-7 in the mean square at
    4), its difference's from the reference (half a step below 8 in powers of four: 2^-22, 1.9e-7), the exponential's and the
    logarithm's (2^-22 and less, 1.5e-7 each), the result's (2^-24 of 7, 2.5e-7 at most): 4e-7 together, half as much again
    allowed."""
    lens = list(range(1, 41))
    Q, codes, scales, table = _make([1] * 40, lens, 16, 4, 64, 16, 26700, spread=0)
    Q[:] = 0
    Q[:, :, 11] = 1.0
    scales[:, 0] = 2.0 ** -6
    codes[:, 0] = codes[:, 0].float().nan_to_num(0).clamp(-256, 256).to(codes.dtype)
    O, LSE = _run(Q, codes, scales, table, [1] * 40, lens, scale=1.0)
    off = []
    for i, n in enumerate(lens):
        k = oracle.kv_cache_rows(f64(codes[:, 0]), f64(scales[:, 0]), table[i].tolist(), 16, 0, n)
        off.append(f64(LSE[:, i]) - np.log(np.exp(np.repeat(k[:, :, 11], 4, axis=1)).sum(0)))
    assert np.sqrt(np.mean(np.square(off))) < 6e-7
