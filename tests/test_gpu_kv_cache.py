"""GPU parity of the 8-bit cache's write and read against the float64 oracle: equal codes, scales and values, bit for bit
(scales are powers of two, so x / scale and code * scale are exact in fp32 and each result is rounded once)."""
import numpy as np
import pytest
import torch

import oracle
import synth
from cache_util import F8, cu_of, f64, ints, page_table, pool
from gpu_util import mp, status_tensor

pytestmark = pytest.mark.gpu


def _write(K, V, codes, scales, table, cu, start, max_n=None, status=0):
    """The write on copies; keys and values of the pool side by side."""
    c, s, st = codes.cuda(), scales.cuda(), status_tensor()
    mp().mp_kv_cache_write(K.cuda(), V.cuda(), c[:, 0], c[:, 1], s[:, 0], s[:, 1], table.cuda(), cu.cuda(), start.cuda(),
                           max_n=int((cu[1:] - cu[:-1]).max()) if max_n is None else max_n, d_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == status
    return c.cpu(), s.cpu()


def _expect(K, V, codes, scales, table, cu, start):
    c, s = f64(codes), f64(scales)
    for i, x in enumerate((K, V)):
        ci, si = c[:, i].copy(), s[:, i].copy()
        oracle.kv_cache_write(f64(x), ci, si, table.numpy(), cu.numpy(), start.numpy(), codes.shape[3])
        c[:, i], s[:, i] = ci, si
    return c, s


def _same(got, want):
    assert np.array_equal(f64(got[1]), want[1], equal_nan=True)
    assert np.array_equal(f64(got[0]), want[0], equal_nan=True)


def _rows(T, kv, d, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(2, T, kv, d, generator=g) * torch.exp(torch.randn(2, T, kv, 1, generator=g))
    return x.to(torch.bfloat16)


CASES = [  # new, start, key heads, d, page
    ([1], [0], 1, 16, 16),
    ([1, 1, 1, 1], [0, 15, 16, 40], 2, 64, 16),          # single tokens: a fresh page, a page's last slot, its first
    ([1] * 70, list(range(0, 210, 3)), 3, 128, 64),      # more sequences than a warp has lanes
    ([5, 0, 33, 17], [0, 9, 31, 100], 2, 96, 32),        # runs that end inside a page, a sequence without rows
    ([300, 1, 64], [0, 63, 64], 2, 80, 64),
    ([130, 127], [127, 1], 1, 256, 128),                 # the widest head, the largest page
    ([37] + [0] * 40 + [2], [3] + [0] * 40 + [14], 5, 48, 16),
    ([1, 999, 3] + [1] * 40, [5, 20, 0] + [7] * 40, 1, 64, 32),  # one long among many single ones: found by the search
]


@pytest.mark.parametrize("new,start,kv,d,page", CASES)
def test_write_matches_oracle(new, start, kv, d, page):
    table, pages = page_table([a + b for a, b in zip(new, start)], page, 22000 + d, room=1)
    codes, scales = pool(pages, kv, page, d, 22001 + d)
    K, V = _rows(sum(new), kv, d, 22002 + page)
    cu, st = cu_of(new), ints(start)
    _same(_write(K, V, codes, scales, table, cu, st), _expect(K, V, codes, scales, table, cu, st))


@pytest.mark.parametrize("new,start,kv,d,page", CASES)
def test_read_matches_oracle(new, start, kv, d, page):
    table, pages = page_table([a + b for a, b in zip(new, start)], page, 22100 + d, room=1)
    codes, scales = pool(pages, kv, page, d, 22101 + d)
    scales *= 1.0 + torch.rand(scales.shape, generator=torch.Generator().manual_seed(7))  # any scales
    c, s, cu, T = codes.cuda(), scales.cuda(), cu_of(new), sum(new)
    out = torch.full((T + 3, 2 * kv, d), 7.0, dtype=torch.bfloat16, device="cuda")
    stat = status_tensor()
    mp().mp_kv_cache_read(c[:, 0], c[:, 1], s[:, 0], s[:, 1], out[:, :kv], out[:, kv:], table.cuda(), cu.cuda(),
                          ints(start).cuda(), max_n=max(new), d_status=stat)
    torch.cuda.synchronize()
    assert int(stat.item()) == 0
    for i in (0, 1):
        want = np.concatenate([oracle.kv_cache_rows(f64(codes[:, i]), f64(scales[:, i]), table[j].tolist(), page, a, n)
                               for j, (a, n) in enumerate(zip(start, new))])
        got = out[:T, i * kv:(i + 1) * kv].cpu()
        assert torch.equal(got, torch.from_numpy(want).float().to(torch.bfloat16))
    assert torch.all(out[T:] == 7.0)  # rows behind the last sequence


def test_token_by_token_then_read_back():
    # scales grow on the way: each value stays within two roundings of its page's scale
    T, kv, d, page = 75, 2, 64, 32
    K, V = _rows(T, kv, d, 22200)
    table, pages = page_table([T], page, 22201)
    codes, scales = pool(pages, kv, page, d, 22202, nan=True)
    c, s = codes.cuda(), scales.cuda()
    want = f64(codes), f64(scales)
    kd, vd, td = K.cuda(), V.cuda(), table.cuda()
    for k in range(T):
        mp().mp_kv_cache_write(kd[k:k + 1], vd[k:k + 1], c[:, 0], c[:, 1], s[:, 0], s[:, 1], td, ints([0, 1]).cuda(),
                               ints([k]).cuda(), max_n=1)
        for i, x in enumerate((K, V)):
            oracle.kv_cache_write(f64(x[k:k + 1]), want[0][:, i], want[1][:, i], table.numpy(), [0, 1], [k], page)
    _same((c.cpu(), s.cpu()), want)
    ko, vo = torch.empty_like(kd), torch.empty_like(vd)
    mp().mp_kv_cache_read(c[:, 0], c[:, 1], s[:, 0], s[:, 1], ko, vo, td, cu_of([T]).cuda(), max_n=T)
    for x, y in ((K, ko), (V, vo)):
        x, y = f64(x), f64(y)
        bound = np.abs(x).max((0, 2), keepdims=True)  # scale <= 2 amax / 448; its smallest step 2^-9, halved, twice
        assert np.all(np.abs(x - y) <= 2.0 ** -4 * np.abs(x) + 2 * 2.0 ** -10 * 2 * bound / 448)


def test_special_values():
    T, kv, d, page = 20, 2, 32, 16
    K, V = _rows(T, kv, d, 22300)
    K[3, 0, 5], K[17, 1, 0], V[0, 0, 0], V[16:, 1] = float("inf"), float("-inf"), float("nan"), 0.0
    V[2, 1, 3] = 3.3e38       # near the largest bf16 value
    K[18, 0] = 1e-38          # far below 2^-100: zeros
    K[16:, 0] = 1e-38
    table, pages = page_table([T + 4], page, 22301)
    codes, scales = pool(pages, kv, page, d, 22302)
    cu, st = cu_of([T]), ints([4])
    # scales that no write leaves: not a power of two, zero, negative, NaN, infinite, and one that is too large
    for before in (0.011, 3.0, 0.0, -1.0, float("nan"), float("inf"), 2.0 ** 121):
        scales[:] = before
        _same(_write(K, V, codes, scales, table, cu, st), _expect(K, V, codes, scales, table, cu, st))


def test_contiguous_pools_and_other_stream():
    T, kv, d, page = 90, 2, 64, 32
    K, V = _rows(T, kv, d, 22400)
    table, pages = page_table([T], page, 22401)
    codes, scales = pool(pages, kv, page, d, 22402)
    want = _write(K, V, codes, scales, table, cu_of([T]), ints([0]))
    dev = [codes[:, 0].contiguous().cuda(), codes[:, 1].contiguous().cuda(), scales[:, 0].contiguous().cuda(),
           scales[:, 1].contiguous().cuda()]
    packed = torch.cat([K, V], 1).cuda()  # rows of one projection
    args = (table.cuda(), cu_of([T]).cuda(), ints([0]).cuda())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    mp().mp_kv_cache_write(packed[:, :kv], packed[:, kv:], *dev, *args, max_n=T + 0, stream=s)
    s.synchronize()
    for i in (0, 1):
        assert torch.equal(dev[i].view(torch.uint8).cpu(), want[0][:, i].contiguous().view(torch.uint8))
        assert torch.equal(dev[2 + i].cpu(), want[1][:, i])


def test_bad_sequences_and_pages_are_left_out():
    kv, d, page = 1, 64, 16
    new = [10, 20, 30, 5]
    K, V = _rows(sum(new), kv, d, 22500)
    table, pages = page_table([n + 8 for n in new], page, 22501)
    codes, scales = pool(pages, kv, page, d, 22502)
    cu, start = cu_of(new), ints([8] * 4)
    whole = _expect(K, V, codes, scales, table, cu, start)

    def check(want, status, **kw):
        a = dict(table=table, cu=cu, start=start)
        a.update({k: v for k, v in kw.items() if k != "max_n"})
        got = _write(K, V, codes, scales, a["table"], a["cu"], a["start"], max_n=kw.get("max_n", 30), status=status)
        _same(got, want)

    def without(i, pages_of=None):
        c, s = whole[0].copy(), whole[1].copy()
        for pg in (table[i].tolist() if pages_of is None else pages_of):
            if pg >= 0:
                c[pg], s[pg] = f64(codes)[pg], f64(scales)[pg]
        return c, s

    check(whole, 0)
    bad = start.clone()
    bad[1] = -1
    check(without(1), 4, start=bad)
    bad[1] = 1 << 30
    check(without(1), 4, start=bad)
    check(without(2), 4, max_n=29)
    bad = table.clone()
    gone = int(bad[2, 1])
    for page_id in (-5, pages, 1 << 30):
        bad[2, 1] = page_id
        check(without(2, [gone]), 8, table=bad)
    # an end behind the rows: the last sequence
    bad = cu.clone()
    bad[4] = sum(new) + 1
    check(without(3), 4, cu=bad)
    # the read leaves the same rows alone
    c, s, st = codes.cuda(), scales.cuda(), status_tensor()
    out = torch.full((sum(new), 2, d), 7.0, dtype=torch.bfloat16, device="cuda")
    bad = table.clone()
    bad[2, 1] = pages
    mp().mp_kv_cache_read(c[:, 0], c[:, 1], s[:, 0], s[:, 1], out[:, :1], out[:, 1:], bad.cuda(), cu.cuda(), start.cuda(),
                          max_n=30, d_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 8
    left = (out == 7.0).all(-1).all(-1).cpu().nonzero()[:, 0].tolist()
    assert left == list(range(30 + 8, 30 + 24))  # slots 0 .. 15 of its second page, positions 16 .. 31


def test_offsets_beyond_32_bits():
    # a pool whose pages lie 2^32 bytes apart in one allocation: 5 pages, 16 GB
    kv, d, page = 1, 64, 16
    apart = 1 << 32
    raw = torch.empty(4 * apart + 2 * page * d, dtype=torch.uint8, device="cuda").view(F8)
    kc = raw.as_strided((5, kv, page, d), (apart, page * d, d, 1))
    vc = raw[page * d:].as_strided((5, kv, page, d), (apart, page * d, d, 1))
    ks, vs = torch.zeros(5, kv, device="cuda"), torch.zeros(5, kv, device="cuda")
    K, V = _rows(70, kv, d, 22600)
    table = ints([4, 1, 3, 0, 2])[None].cuda()
    cu, start = cu_of([70]).cuda(), ints([5]).cuda()
    for x in (kc, vc):
        for i in range(5):
            x[i].view(torch.uint8).zero_()
    ks.fill_(2.0 ** -6)
    vs.fill_(2.0 ** -6)
    mp().mp_kv_cache_write(K.cuda(), V.cuda(), kc, vc, ks, vs, table, cu, start, max_n=70)
    codes, scales = torch.zeros(5, 2, kv, page, d).to(F8), torch.full((5, 2, kv), 2.0 ** -6)
    want = _expect(K, V, codes, scales, table.cpu(), cu.cpu(), start.cpu())
    for i, (c, s) in enumerate(((kc, ks), (vc, vs))):
        got = torch.stack([c[k].view(torch.uint8) for k in range(5)]).view(F8)
        assert np.array_equal(f64(got), want[0][:, i]) and np.array_equal(f64(s), want[1][:, i])
    ko, vo = torch.empty(70, kv, d, dtype=torch.bfloat16, device="cuda"), torch.empty(70, kv, d, dtype=torch.bfloat16,
                                                                                      device="cuda")
    mp().mp_kv_cache_read(kc, vc, ks, vs, ko, vo, table, cu, start, max_n=70)
    rows = oracle.kv_cache_rows(want[0][:, 1], want[1][:, 1], [4, 1, 3, 0, 2], page, 5, 70)
    assert np.array_equal(f64(vo), rows)
