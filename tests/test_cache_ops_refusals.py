"""What the query and key norm, the 8-bit cache and the attention over it refuse, before any CUDA work (CPU only)."""
import ctypes

import pytest
import torch

FAKE = ctypes.c_void_p(0x100000)   # never dereferenced
BAD = ctypes.c_void_p(0x100002)
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    from tensor_transformer_layer_gb300 import build
    build.build()
    import tensor_transformer_layer_gb300 as mp
    return mp.lib()


def _norm(L, x=FAKE, y=FAKE, wq=FAKE, wk=FAKE, pos=FAKE, T=8, heads=4, nq=3, d=64, ldx=None, ldy=None, sections=(16, 8, 8),
          base=1e4, eps=1e-6, flags=0, axes=None):
    sec = (ctypes.c_int * max(len(sections), 1))(*sections)
    ldx, ldy = (heads * d if v is None else v for v in (ldx, ldy))
    axes = len(sections) if axes is None else axes
    fwd = L.mp_qk_norm_rope(x, y, wq, wk, pos, T, heads, nq, d, ldx, ldy, axes, sec, base, eps, flags, None)
    other = ctypes.c_void_p(0x900000)
    bwd = L.mp_qk_norm_rope_bwd(x, other, y, wq, wk, FAKE, FAKE, pos, FAKE, BIG, T, heads, nq, d, ldx, heads * d, ldy, axes,
                                sec, base, eps, flags, None)
    if T > 0:
        assert fwd == bwd
    return fwd


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 1), (dict(heads=0), 1), (dict(nq=-1), 1), (dict(nq=5), 1), (dict(d=0), 1), (dict(axes=0), 1),
    (dict(sections=(8,) * 5), 1), (dict(sections=(16, -8, 8)), 1), (dict(base=0.0), 1), (dict(base=float("nan")), 1),
    (dict(eps=0.0), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(flags=4), 1), (dict(flags=8), 1),          # the inverse is the backward pass's
    (dict(d=60), 2), (dict(d=264, sections=(16,)), 2), (dict(sections=(0, 0)), 2), (dict(sections=(3, 3)), 2),
    (dict(sections=(32, 4)), 2), (dict(ldx=255), 2), (dict(ldy=248), 2), (dict(ldx=260), 2),
    (dict(x=None), 1), (dict(y=None), 1), (dict(pos=None), 1), (dict(wq=None), 1), (dict(wk=None), 1),
    (dict(x=BAD), 3), (dict(y=BAD), 3), (dict(pos=BAD), 3), (dict(wq=BAD), 3), (dict(wk=BAD), 3),
    (dict(ldx=320), 1),   # in place with two pitches
])
def test_norm_refusals(L, kw, code):
    assert _norm(L, **kw) == code


def test_norm_backward_refusals(L):
    sec = (ctypes.c_int * 1)(32)

    def bwd(dwq=FAKE, dwk=FAKE, ws=FAKE, wb=BIG, T=8, dy=ctypes.c_void_p(0x900000), lddy=256):
        return L.mp_qk_norm_rope_bwd(FAKE, dy, FAKE, FAKE, FAKE, dwq, dwk, FAKE, ws, wb, T, 4, 3, 64, 256, lddy, 256, 1, sec,
                                     1e4, 1e-6, 0, None)

    need = L.mp_qk_norm_rope_bwd_workspace_bytes(8, 4, 64)
    assert need > 0 and need % (2 * 64 * 4) == 0
    assert bwd(dwq=None) == 1 and bwd(dwk=None) == 1 and bwd(dwq=None, T=0) == 1
    assert bwd(dwq=BAD) == 3 and bwd(dy=None) == 1 and bwd(dy=BAD) == 3 and bwd(lddy=252) == 2
    assert bwd(ws=None) == 8 and bwd(ws=BAD) == 8 and bwd(wb=need - 1) == 8
    assert bwd(dy=FAKE, lddy=320) == 1   # dx is dy with another pitch
    for T, heads, d in ((0, 4, 64), (-1, 4, 64), (8, 0, 64), (8, 4, 60), (8, 4, 264)):
        assert L.mp_qk_norm_rope_bwd_workspace_bytes(T, heads, d) == 0


def test_norm_empty_batch_is_a_noop(L):
    assert _norm(L, x=None, y=None, wq=None, wk=None, pos=None, T=0) == 0


def _kv(L, K=FAKE, V=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, table=FAKE, cu=FAKE, start=FAKE, nseq=2, T=100, max_n=60,
        kv=2, d=64, page=32, pages=9, max_pages=4, ldk=None, ldv=None, ldkc=None, ldvc=None, ldks=None, ldvs=None, st=None):
    row, run = kv * d, kv * d * page
    rest = (nseq, T, max_n, kv, d, page, pages, max_pages, row if ldk is None else ldk, row if ldv is None else ldv,
            run if ldkc is None else ldkc, run if ldvc is None else ldvc, kv if ldks is None else ldks,
            kv if ldvs is None else ldvs, st, None)
    w = L.mp_kv_cache_write(K, V, kc, vc, ks, vs, table, cu, start, *rest)
    r = L.mp_kv_cache_read(kc, vc, ks, vs, K, V, table, cu, start, *rest)
    assert w == r or start is None
    return w


POOL_REFUSALS = [
    (dict(nseq=-1), 1), (dict(kv=0), 1), (dict(d=0), 1), (dict(pages=-1), 1), (dict(max_pages=-1), 1),
    (dict(page=8), 2), (dict(page=48), 2), (dict(page=256), 2), (dict(pages=0), 2), (dict(max_pages=0), 2),
    (dict(max_pages=1 << 27), 2), (dict(ldkc=4080), 2), (dict(ldvc=4080), 2), (dict(ldkc=4104), 2), (dict(ldvc=4104), 2),
    (dict(ldks=1), 2), (dict(ldvs=1), 2), (dict(kc=None), 1), (dict(vc=None), 1), (dict(ks=None), 1), (dict(vs=None), 1),
    (dict(table=None), 1), (dict(kc=BAD), 3), (dict(vc=BAD), 3), (dict(ks=BAD), 3), (dict(vs=BAD), 3), (dict(table=BAD), 3),
    (dict(cu=None), 1), (dict(cu=BAD), 3), (dict(st=BAD), 3),
]


@pytest.mark.parametrize("kw,code", POOL_REFUSALS + [
    (dict(T=-1), 1), (dict(max_n=-1), 1), (dict(max_n=101), 2), (dict(d=72), 2), (dict(d=272), 2), (dict(ldk=120), 2),
    (dict(ldk=1 << 28), 2), (dict(ldv=1 << 28), 2), (dict(ldv=132), 2), (dict(K=None), 1), (dict(V=None), 1), (dict(start=None), 1), (dict(K=BAD), 3), (dict(V=BAD), 3),
    (dict(start=BAD), 3),
    (dict(nseq=0x7fffffff, T=0x7fffffff, max_n=33), 2),   # more pages than a grid has CTAs
])
def test_cache_refusals(L, kw, code):
    assert _kv(L, **kw) == code


def test_cache_without_rows_is_a_noop(L):
    assert _kv(L, nseq=0, K=None, cu=None) == 0 and _kv(L, max_n=0, K=None, kc=None) == 0


def _attn(L, Q=FAKE, O=FAKE, LSE=FAKE, lens=FAKE, cu=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, table=FAKE, ws=FAKE, wb=BIG,
          nseq=2, Tq=20, max_q=4, heads=4, kv=2, d=64, page=32, pages=9, max_pages=4, ldq=None, ldo=None, ldkc=None,
          ldvc=None, ldks=None, ldvs=None, scale=0.125, st=None):
    row, run = heads * d, kv * d * page
    return L.mp_attn_cache_fwd(Q, kc, vc, ks, vs, O, LSE, table, cu, lens, ws, wb, nseq, Tq, max_q, heads, kv, d, page,
                               pages, max_pages, row if ldq is None else ldq, row if ldo is None else ldo,
                               run if ldkc is None else ldkc, run if ldvc is None else ldvc, kv if ldks is None else ldks,
                               kv if ldvs is None else ldvs, 1, scale, st, None)


@pytest.mark.parametrize("kw,code", POOL_REFUSALS + [
    (dict(Tq=-1), 1), (dict(max_q=-1), 1), (dict(heads=0), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(d=80), 2), (dict(d=256), 2), (dict(heads=3), 2),
    (dict(max_q=21), 2), (dict(heads=131072), 2), (dict(ldq=248), 2), (dict(ldo=260), 2), (dict(Tq=1 << 30, max_q=1 << 29), 2),
    (dict(Q=None), 1), (dict(O=None), 1), (dict(LSE=None), 1), (dict(lens=None), 1), (dict(Q=BAD), 3), (dict(O=BAD), 3),
    (dict(LSE=BAD), 3), (dict(lens=BAD), 3), (dict(ws=None), 8), (dict(ws=BAD), 8), (dict(wb=4096), 8),
])
def test_attention_refusals(L, kw, code):
    assert _attn(L, **kw) == code


def test_attention_without_queries_is_a_noop(L):
    assert _attn(L, nseq=0, Q=None) == 0 and _attn(L, max_q=0, cu=None, ws=None) == 0


def test_attention_workspace_bytes(L):
    w = L.mp_attn_cache_workspace_bytes
    assert 0 < w(16, 4, 96, 1) <= w(16, 4, 96, 9) <= w(16, 4, 128, 9)
    for a in ((0, 1, 64, 1), (4, 0, 64, 1), (4, 3, 64, 1), (4, 2, 80, 1), (4, 2, 64, 0)):
        assert w(*a) == 0


def test_status_names(L):
    import tensor_transformer_layer_gb300 as mp
    assert mp.mp_status_from_device(mp.MP_DEV_PAGE_RANGE) == 10
    assert mp.status_string(10).startswith(mp.STATUS_NAMES[10])


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device answer")
def test_no_device_answer(L):
    assert _norm(L) == 4 and _kv(L) == 4 and _attn(L) == 4


def test_binding_refusals():
    import tensor_transformer_layer_gb300 as mp
    x, w = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16)
    pos, f = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(64)
    u8 = torch.zeros(64, dtype=torch.uint8)
    how = dict(q_heads=1, sections=(32,))
    with pytest.raises(ValueError, match="CUDA"):
        mp.mp_qk_norm_rope(x, x, w, w, pos, **how)
    with pytest.raises(ValueError, match="3|tokens"):
        mp.mp_qk_norm_rope(x[0], x[0], w, w, pos, **how)
    with pytest.raises(ValueError, match="32 bits"):
        mp.mp_qk_norm_rope(x, x, w, w, pos, q_heads=1 << 32, sections=(32,))
    with pytest.raises(ValueError):
        mp.mp_qk_norm_rope_bwd(x, x, x, w, w, f, f, pos, u8, **how)
    with pytest.raises(TypeError):
        mp._page_view(x[0], "ks", torch.float32, x[0].shape, [1])
    codes = torch.zeros(5, 2, 2, 16, 64).to(torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="contiguous"):
        mp._page_view(codes[..., ::2], "kc", codes.dtype, codes[..., ::2].shape, [512, 256, 32, 1])
    scales = torch.ones(5, 2, 2)
    pool = (codes[:, 0], codes[:, 1], scales[:, 0], scales[:, 1])
    table, cu = torch.zeros(1, 2, dtype=torch.int32), torch.tensor([0, 4], dtype=torch.int32)
    start = torch.zeros(1, dtype=torch.int32)
    for bad, why in (((codes[0, 0], *pool[1:]), ValueError),
                     ((*pool[:2], scales[:, 0].double(), pool[3]), TypeError),
                     ((*pool[:3], scales[:4, 1]), ValueError), ((*pool[:2], None, pool[3]), TypeError),
                     (pool, ValueError)):     # the last: not on the GPU
        with pytest.raises(why):
            mp._pool(*bad, table, 1)
    for call in (lambda: mp.mp_kv_cache_write(x, x, *pool, table, cu, start, max_n=4),
                 lambda: mp.mp_kv_cache_read(*pool, x, x, table, cu, max_n=4),
                 lambda: mp.mp_attn_cache_fwd(x, *pool, x, torch.zeros(2, 4), table, cu, start, u8, max_q=4)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="32 bits"):
        mp.mp_attn_cache_workspace_bytes(1 << 32, 1, 64, 1)
