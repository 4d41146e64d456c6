"""GPU parity of the attention over the 8-bit cache against the float64 oracle.

Tolerance per element of O: half a bf16 step of the result (2^-8), the probabilities' rounding to halves (2^-11 of each,
at least 2^-32 of the largest) and the scores' error, relative to A = sum P |v|. A score is a sum of d fp32 products of
magnitudes S' = scale sum |q k|: 2^-20 S', and ex2 and the factors add 2^-20. The log-sum-exp: the score's error, and its own
roundings, 2^-21 of it and of one."""
import numpy as np
import pytest
import torch

import oracle
import synth
from cache_util import cu_of, f64, ints, page_table, pool
from gpu_util import mp, status_tensor

pytestmark = pytest.mark.gpu


def _nan(*shape, dtype=torch.bfloat16):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def _make(new, lens, heads, kv, d, page, seed, spread=2, q=1.0):
    """Queries and a pool that holds NaN wherever no sequence has a token."""
    table, pages = page_table(lens, page, seed, room=1)
    codes, scales = pool(pages, kv, page, d, seed + 1, spread)
    raw = codes.view(torch.uint8)
    mine = torch.zeros(pages, page, dtype=torch.bool)
    for i, n in enumerate(lens):
        for j in range(0, n, page):
            mine[table[i, j // page], :min(page, n - j)] = True
    raw.copy_(torch.where(mine[:, None, None, :, None], raw, torch.tensor(0x7f, dtype=torch.uint8)))
    scales[~mine[:, 0]] = float("nan")
    Q = (synth.normal_bf16((sum(new), heads, d), 1.0, seed + 2).float() * q).to(torch.bfloat16)
    return Q, codes, scales, table


def _workspace(heads, kv, d, max_q):
    """Full of NaN: nothing in it needs to be set before a call."""
    return torch.full((mp().mp_attn_cache_workspace_bytes(heads, kv, d, max_q),), 0xff, dtype=torch.uint8, device="cuda")


def _run(Q, codes, scales, table, new, lens, causal=True, scale=None, status=0, max_q=None, cu=None, ws=None):
    T, heads, d = Q.shape
    kv = codes.shape[2]
    c, s, st = codes.cuda(), scales.cuda(), status_tensor()
    mq = max(new) if max_q is None else max_q
    ws = _workspace(heads, kv, d, mq) if ws is None else ws
    O, LSE = _nan(T, heads, d), _nan(heads, T, dtype=torch.float32)
    mp().mp_attn_cache_fwd(Q.cuda(), c[:, 0], c[:, 1], s[:, 0], s[:, 1], O, LSE, table.cuda(),
                           (cu_of(new) if cu is None else cu).cuda(), ints(lens).cuda(), ws, max_q=mq, causal=causal,
                           scale=scale, d_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == status, int(st.item())
    return O.cpu(), LSE.cpu()


def _check(got, Q, codes, scales, table, new, lens, causal=True, scale=None, skip=None):
    O, LSE = f64(got[0]), f64(got[1])
    heads, d, kv, page = Q.shape[1], Q.shape[2], codes.shape[2], codes.shape[3]
    scale = d ** -0.5 if scale is None else scale
    q, row = f64(Q), 0
    for i, (nq, nk) in enumerate(zip(new, lens)):
        k, v = (oracle.kv_cache_rows(f64(codes[:, j]), f64(scales[:, j]), table[i].tolist(), page, 0, nk) for j in (0, 1))
        at = slice(row, row + nq)
        row += nq
        if i == skip:
            continue
        wo, wl = oracle.attn_varlen_fwd(q[at], k, v, [0, nq], [0, nk], causal, scale)
        wa, _ = oracle.attn_varlen_fwd(q[at], k, np.abs(v), [0, nq], [0, nk], causal, scale)
        seen = np.isfinite(wl)
        assert np.array_equal(np.isfinite(LSE[:, at]), seen) and not np.isnan(LSE[:, at]).any()
        assert not O[at][~seen.T].any()
        if nk == 0 or nq == 0:
            continue
        kk = np.repeat(np.abs(k), heads // kv, axis=1)
        most = scale * np.einsum("qhd,khd->hqk", np.abs(q[at]), kk).max(-1)  # [heads, nq]
        es = 2.0 ** -20 * most + 2.0 ** -20
        vmax = np.repeat(np.abs(v).max((0, 2)), heads // kv)
        tol = (2.0 ** -8 * np.abs(wo) + (2.0 ** -11 + 2 * es.T[..., None]) * wa
               + 2.0 ** -32 * nk * vmax[None, :, None])
        err = np.abs(O[at] - wo) - tol
        assert np.all(err <= 0), (i, float(err.max()))
        le = np.abs(LSE[:, at][seen] - wl[seen]) - (es[seen] + 2.0 ** -21 * (1 + np.abs(wl[seen])))
        assert np.all(le <= 0), (i, float(le.max()))


CASES = [  # new, lens, heads, key heads, d, page
    ([1], [1], 1, 1, 64, 16),                       # one token that sees itself
    ([1], [16], 2, 1, 96, 16),
    ([1], [33], 8, 1, 128, 32),                     # a tile and a token
    ([1, 1, 1], [31, 64, 129], 8, 2, 128, 64),
    ([1] * 9, [0, 1, 15, 16, 17, 47, 48, 49, 300], 6, 2, 64, 16),   # pages that end inside a tile; an empty cache
    ([1] * 9, [0, 1, 31, 32, 33, 127, 128, 129, 1000], 16, 4, 96, 128),
    ([1], [5000], 16, 2, 128, 64),                  # one long sequence: split among the CTAs
    ([1, 1], [20000, 3], 8, 1, 64, 32),
    ([1], [7777], 5, 5, 96, 16),                    # a query head to each key head
    ([4, 6, 1, 5], [1000, 3, 40, 0], 16, 4, 64, 16),   # 16 and 24 rows; rows that see nothing
    ([3, 0, 2], [2500, 100, 2], 12, 1, 128, 32),    # 36 rows of one key head; a sequence without queries
    ([70, 33], [700, 50], 4, 2, 96, 64),            # a chunk of a prompt, longer than its cache in the second
    ([1] * 300, [(i * 37) % 97 for i in range(300)], 2, 1, 64, 16),  # more sequences than the block has threads
    ([1] * 40, [200 + i for i in range(40)], 64, 8, 128, 128),
    ([(i % 5 + 1) // 2 for i in range(1100)], [(i * 37) % 41 for i in range(1100)], 2, 1, 64, 16),  # several steps of a search
    ([2, 5], [400, 90], 36, 3, 64, 32),             # twelve heads of a group: queries begin inside a row tile
]


@pytest.mark.parametrize("new,lens,heads,kv,d,page", CASES)
@pytest.mark.parametrize("causal", [True, False])
def test_matches_oracle(new, lens, heads, kv, d, page, causal):
    inp = _make(new, lens, heads, kv, d, page, 23000 + d + page + len(new))
    _check(_run(*inp, new, lens, causal), *inp, new, lens, causal)


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("rows", [1, 8, 9, 16, 17, 33])
def test_every_width_at_row_counts_around_a_tile(d, rows):
    new, lens = [rows, 1], [rows + 200, 777]
    inp = _make(new, lens, 1, 1, d, 32, 23200 + rows)
    _check(_run(*inp, new, lens), *inp, new, lens)


def test_repeats_bit_for_bit_with_one_workspace_for_other_sizes():
    ws = _workspace(16, 1, 128, 4)
    a = _make([1, 1], [3000, 900], 16, 2, 128, 64, 23300)
    b = _make([4], [6000], 12, 1, 64, 16, 23301)
    first = _run(*a, [1, 1], [3000, 900], ws=ws)
    other = _run(*b, [4], [6000], ws=ws)
    for _ in range(3):
        for inp, want, new, lens in ((a, first, [1, 1], [3000, 900]), (b, other, [4], [6000])):
            got = _run(*inp, new, lens, ws=ws)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_scales_far_apart():
    # pages whose scales differ by 2^40, among them zero pages at the smallest scale
    inp = _make([1, 2], [500, 300], 4, 2, 64, 16, 23400, spread=20, q=2.0 ** -18)
    Q, codes, scales, table = inp
    pg = int(table[0, 3])
    codes.view(torch.uint8)[pg] = 0
    scales[pg] = 2.0 ** -100
    first = int(table[1, 0])
    codes.view(torch.uint8)[first, 1] = 0
    scales[first, 1] = 0.0
    _check(_run(*inp, [1, 2], [500, 300]), *inp, [1, 2], [500, 300])


def test_scales_below_the_normal_numbers():
    """Value scales that no write leaves: results of 1e-36 and less keep what bf16 holds of them. Halves below 2^-14 add
    2^-25 of 2^-120 a token (P carries 2^7), bf16 half its least step, 2^-134."""
    new, lens = [1, 2, 1], [300, 90, 40]
    Q, codes, scales, table = _make(new, lens, 4, 2, 64, 16, 23450)
    for i, n in enumerate(lens):
        for j in range(0, n, 16):
            if i != 1 or j % 32 == 0:  # the second sequence has ordinary pages between
                scales[int(table[i, j // 16]), 1] = (2.0 ** -121, 2.0 ** -127, 2.0 ** -135, 1.4e-45)[j // 16 % 4]
    O, LSE = _run(Q, codes, scales, table, new, lens)
    row = 0
    for i, (nq, nk) in enumerate(zip(new, lens)):
        k, v = (oracle.kv_cache_rows(f64(codes[:, j]), f64(scales[:, j]), table[i].tolist(), 16, 0, nk) for j in (0, 1))
        at = slice(row, row + nq)
        row += nq
        wo, wl = oracle.attn_varlen_fwd(f64(Q)[at], k, v, [0, nq], [0, nk], True, 0.125)
        wa, _ = oracle.attn_varlen_fwd(f64(Q)[at], k, np.abs(v), [0, nq], [0, nk], True, 0.125)
        small = nk * 2.0 ** -152 * 448 + 2.0 ** -134
        big = 2.0 ** -32 * nk * np.abs(v).max()
        assert np.all(np.abs(f64(O)[at] - wo) <= 2.0 ** -8 * np.abs(wo) + 2.0 ** -9 * wa + small + big), i
        assert np.all(np.abs(f64(LSE)[:, at] - wl) <= 2.0 ** -12 * (1 + np.abs(wl)))


def test_scales_that_are_no_powers_of_two_and_large_queries():
    Q, codes, scales, table = _make([1, 3], [700, 200], 8, 2, 96, 32, 23500)
    scales *= 1.0 + torch.rand(scales.shape, generator=torch.Generator().manual_seed(5))
    Q[0, 0, 0], Q[0, 1], Q[1, 2] = 3e38, 1e-38, 0.0
    Q[2] *= 30  # scores of a few hundred
    _check(_run(Q, codes, scales, table, [1, 3], [700, 200], scale=0.01), Q, codes, scales, table, [1, 3], [700, 200],
           scale=0.01)


def test_scores_that_rise_along_the_cache():
    # each tile's largest score passes the last one's by more than the slack: sums are scaled down again and again
    new, lens, heads, kv, d, page = [1, 1], [900, 257], 8, 1, 64, 32
    Q, codes, scales, table = _make(new, lens, heads, kv, d, page, 23600)
    for i, n in enumerate(lens):
        for j in range(n):
            codes[int(table[i, j // page]), 0, :, j % page] = (j // 7 % 200) * 1.0
    scales[:] = 2.0 ** -4
    Q[:] = Q.abs()
    _check(_run(Q, codes, scales, table, new, lens, scale=0.5), Q, codes, scales, table, new, lens, scale=0.5)


def test_nan_and_infinite_queries_stay_in_their_rows():
    new, lens = [1, 1, 2], [300, 40, 90]
    Q, codes, scales, table = _make(new, lens, 4, 1, 64, 16, 23700)
    clean = _run(Q, codes, scales, table, new, lens)
    Q[0, 1, 3], Q[2, 0, 7] = float("nan"), float("inf")
    O, LSE = _run(Q, codes, scales, table, new, lens)
    hit = torch.zeros(4, 4, dtype=torch.bool)
    hit[0, 1] = hit[2, 0] = True
    assert torch.equal(torch.isnan(O).all(-1), hit)
    assert torch.isnan(LSE.t()[0, 1])
    assert torch.equal(O[~hit], clean[0][~hit]) and torch.equal(LSE.t()[~hit], clean[1].t()[~hit])


def test_nan_in_the_cache_reaches_the_rows_that_see_it():
    new, lens = [2, 1], [200, 70]
    Q, codes, scales, table = _make(new, lens, 2, 2, 64, 16, 23800)
    clean = _run(Q, codes, scales, table, new, lens)
    codes.view(torch.uint8)[int(table[0, 199 // 16]), 0, 0, 199 % 16, 3] = 0x7f  # a key that the last query alone sees
    O, LSE = _run(Q, codes, scales, table, new, lens)
    assert torch.isnan(O[1, 0]).all() and torch.isnan(LSE[0, 1])
    keep = torch.ones(3, 2, dtype=torch.bool)
    keep[1, 0] = False
    assert torch.equal(O[keep], clean[0][keep]) and torch.equal(LSE.t()[keep], clean[1].t()[keep])


def test_bad_sequences_and_pages():
    new, lens = [1, 2, 1], [100, 50, 60]
    Q, codes, scales, table = _make(new, lens, 4, 2, 64, 16, 23900)

    def rows_left(got, lo, hi):
        # The others by their own tolerance: how the work is split, and so the order of sums, goes by all sequences.
        assert torch.isnan(got[0][lo:hi]).all() and torch.isnan(got[1][:, lo:hi]).all()
        _check(got, Q, codes, scales, table, new, lens, skip=1 if lo == 1 else 2)

    for bad in (-1, table.shape[1] * 16 + 1):
        rows_left(_run(Q, codes, scales, table, new, [100, bad, 60], status=4), 1, 3)
    rows_left(_run(Q, codes, scales, table, new, lens, max_q=1, status=4), 1, 3)
    rows_left(_run(Q, codes, scales, table, new, lens, status=4, cu=ints([0, 1, 3, 9])), 3, 4)
    for page_id in (-7, codes.shape[0], 1 << 30):
        t = table.clone()
        t[1, 2] = page_id
        rows_left(_run(Q, codes, scales, t, new, lens, status=8), 1, 3)
    # nothing to do
    assert torch.isnan(_run(Q, codes, scales, table, [0, 0, 0], lens, max_q=1)[0]).all()


def test_strided_rows_contiguous_pools_and_replayed_graph():
    new, lens, heads, kv, d = [1, 1, 1], [4000, 17, 333], 8, 2, 96
    Q, codes, scales, table = _make(new, lens, heads, kv, d, 32, 24000)
    want = _run(Q, codes, scales, table, new, lens)
    dev = [codes[:, 0].contiguous().cuda(), codes[:, 1].contiguous().cuda(), scales[:, 0].contiguous().cuda(),
           scales[:, 1].contiguous().cuda()]
    rows, out = torch.zeros(3, heads + 3, d, dtype=torch.bfloat16, device="cuda"), _nan(3, heads + 1, d)
    rows[:, 2:2 + heads] = Q.cuda()
    LSE, ws = _nan(heads, 3, dtype=torch.float32), _workspace(heads, kv, d, 1)
    args = (table.cuda(), cu_of(new).cuda(), ints(lens).cuda(), ws)

    def call(**kw):
        mp().mp_attn_cache_fwd(rows[:, 2:2 + heads], *dev, out[:, :heads], LSE, *args, max_q=1, **kw)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call(stream=s)
    s.synchronize()
    assert torch.equal(out[:, :heads].cpu(), want[0]) and torch.equal(LSE.cpu(), want[1])
    assert torch.isnan(out[:, heads:]).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
        call()
    for _ in range(3):
        out.fill_(float("nan"))
        LSE.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[:, :heads].cpu(), want[0]) and torch.equal(LSE.cpu(), want[1])


def test_sequences_share_pages_and_rows_of_no_sequence_stay():
    # the second sequence's cache begins with the first one's pages; rows before and behind the sequences are left alone
    lens, new = [150, 200], [2, 1]
    Q, codes, scales, table = _make(new, lens, 4, 2, 64, 32, 24200)
    table[1, :4] = table[0, :4]
    T = 7
    wide = torch.zeros(T, 4, 64, dtype=torch.bfloat16)
    wide[2:5] = Q
    O, LSE = _run(wide, codes, scales, table, new, lens, cu=ints([2, 4, 5]))
    assert torch.isnan(O[[0, 1, 5, 6]]).all() and torch.isnan(LSE[:, [0, 1, 5, 6]]).all()
    _check((O[2:5], LSE[:, 2:5]), Q, codes, scales, table, new, lens)


def test_two_streams_with_a_workspace_each():
    args = []
    for k, (new, lens) in enumerate((([1, 1], [9000, 40]), ([3], [5000]))):
        inp = _make(new, lens, 8, 2, 128, 64, 24300 + k)
        args.append((inp, new, lens, _run(*inp, new, lens)))
    dev, outs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for (Q, codes, scales, table), new, lens, _ in args:
        c, s = codes.cuda(), scales.cuda()
        dev.append((Q.cuda(), c[:, 0], c[:, 1], s[:, 0], s[:, 1], table.cuda(), cu_of(new).cuda(), ints(lens).cuda(),
                    _workspace(8, 2, 128, max(new)), max(new)))
    torch.cuda.synchronize()
    for rep in range(20):
        for (Q, kc, vc, ks, vs, table, cu, ln, ws, mq), st in zip(dev, streams):
            O, LSE = torch.empty_like(Q), torch.empty(8, Q.shape[0], device="cuda")
            st.wait_stream(torch.cuda.current_stream())
            mp().mp_attn_cache_fwd(Q, kc, vc, ks, vs, O, LSE, table, cu, ln, ws, max_q=mq, stream=st)
            outs.append((O, LSE))
    torch.cuda.synchronize()
    for i, (O, LSE) in enumerate(outs):
        want = args[i % 2][3]
        assert torch.equal(O.cpu(), want[0]) and torch.equal(LSE.cpu(), want[1])


def test_decoding_steps_agree_with_the_whole_prompt():
    """A layer's operators as they are used: norm and rotation, write, attention over the cache; a prompt, then single
    tokens and a draft of three, against the packed attention over what the cache holds at each step."""
    heads, kv, d, page, sec = 8, 2, 64, 32, (32,)
    lens, steps = [70, 5], [[1, 1], [1, 1], [3, 3], [1, 0]]
    total = [n + sum(s[i] for s in steps) for i, n in enumerate(lens)]
    table, pages = page_table(total, page, 24100)
    codes, scales = pool(pages, kv, page, d, 24101, nan=True)
    c, s, td = codes.cuda(), scales.cuda(), table.cuda()
    w = (1 + 0.1 * torch.randn(2, d, generator=torch.Generator().manual_seed(3))).to(torch.bfloat16).cuda()
    ws = _workspace(heads, kv, d, 70)
    at = [0, 0]
    for k, new in enumerate([lens] + steps):
        T = sum(new)
        qkv = synth.normal_bf16((T, heads + 2 * kv, d), 1.0, 24110 + k).cuda()
        pos = ints(a + j for a, n in zip(at, new) for j in range(n))[None].cuda()
        cu, start = cu_of(new).cuda(), ints(at).cuda()
        mp().mp_qk_norm_rope(qkv[:, :heads + kv], qkv[:, :heads + kv], w[0], w[1], pos, q_heads=heads, sections=sec)
        mp().mp_kv_cache_write(qkv[:, heads:heads + kv], qkv[:, heads + kv:], c[:, 0], c[:, 1], s[:, 0], s[:, 1], td, cu,
                               start, max_n=max(new))
        at = [a + n for a, n in zip(at, new)]
        O, LSE = _nan(T, heads, d), _nan(heads, T, dtype=torch.float32)
        mp().mp_attn_cache_fwd(qkv[:, :heads], c[:, 0], c[:, 1], s[:, 0], s[:, 1], O, LSE, td, cu, ints(at).cuda(), ws,
                               max_q=max(new))
        ko, vo = torch.empty(sum(at), kv, d, dtype=torch.bfloat16, device="cuda"), torch.empty(
            sum(at), kv, d, dtype=torch.bfloat16, device="cuda")
        mp().mp_kv_cache_read(c[:, 0], c[:, 1], s[:, 0], s[:, 1], ko, vo, td, cu_of(at).cuda(), max_n=max(at))
        O2, LSE2 = _nan(T, heads, d), _nan(heads, T, dtype=torch.float32)
        mp().mp_attn_varlen_fwd(qkv[:, :heads], ko, vo, O2, LSE2, cu, cu_of(at).cuda(), max_q=max(new), max_k=max(at),
                                causal=True)
        # the packed attention rounds its probabilities to bf16 (2^-8), both round O: 3 half steps, and the values' sum
        A = _nan(T, heads, d)
        mp().mp_attn_varlen_fwd(qkv[:, :heads], ko, vo.abs(), A, LSE2.clone(), cu, cu_of(at).cuda(), max_q=max(new),
                                max_k=max(at), causal=True)
        torch.cuda.synchronize()
        err = (O.double() - O2.double()).abs() - 2.0 ** -7 * O2.double().abs() - 1.2 * 2.0 ** -8 * A.double()
        assert float(err.max()) <= 0, k
        assert float((LSE - LSE2).abs().max()) < 2e-4
