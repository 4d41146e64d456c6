"""What the rotation, the gated block and the packed attention refuse, before any CUDA work (CPU only)."""
import ctypes

import pytest
import torch

FAKE = ctypes.c_void_p(0x100000)   # never dereferenced
BAD = ctypes.c_void_p(0x100002)


@pytest.fixture(scope="module")
def L():
    from tensor_transformer_layer_gb300 import build
    build.build()
    import tensor_transformer_layer_gb300 as mp
    return mp.lib()


def _glu(L, T=8, h=64, f=128, t=1, act=0, X=FAKE, Z=FAKE, GU=None):
    fwd = L.mp_glu_fwd(X, FAKE, FAKE, Z, FAKE, GU, T, h, f, t, act, None, None)
    bwd = L.mp_glu_bwd(X, FAKE, FAKE, FAKE, FAKE, FAKE, Z, FAKE, FAKE, FAKE, T, h, f, t, act, None, None)
    assert fwd == bwd
    return fwd


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 1), (dict(h=0), 1), (dict(f=0), 1), (dict(t=0), 1), (dict(act=2), 1), (dict(act=-1), 1),
    (dict(h=96), 2), (dict(f=192, t=2), 2), (dict(t=3), 2), (dict(f=1 << 30), 2),
    (dict(X=None), 1), (dict(Z=None), 1), (dict(X=BAD), 3), (dict(Z=BAD), 3),
])
def test_glu_refusals(L, kw, code):
    assert _glu(L, **kw) == code


def test_glu_empty_batch_is_a_noop(L):
    assert L.mp_glu_fwd(None, None, None, None, None, None, 0, 64, 128, 2, 0, None, None) == 0
    assert L.mp_glu_fwd(FAKE, FAKE, FAKE, FAKE, FAKE, BAD, 8, 64, 128, 2, 0, None, None) == 3
    # the weights' gradients are written even then
    assert L.mp_glu_bwd(None, FAKE, FAKE, None, None, None, None, None, FAKE, None, 0, 64, 128, 2, 0, None, None) == 1


def _rope(L, x=FAKE, y=FAKE, pos=FAKE, T=8, heads=4, d=64, ldx=None, ldy=None, sections=(16, 8, 8), base=1e4, flags=0,
          axes=None):
    sec = (ctypes.c_int * max(len(sections), 1))(*sections)
    return L.mp_rope_axes(x, y, pos, T, heads, d, heads * d if ldx is None else ldx, heads * d if ldy is None else ldy,
                          len(sections) if axes is None else axes, sec, base, flags, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 1), (dict(heads=0), 1), (dict(d=0), 1), (dict(axes=0), 1), (dict(sections=(8,) * 5), 1),
    (dict(sections=(16, -8, 8)), 1), (dict(base=0.0), 1), (dict(base=-2.0), 1), (dict(base=float("nan")), 1),
    (dict(base=float("inf")), 1), (dict(flags=8), 1),
    (dict(d=60), 2), (dict(d=264, sections=(16,)), 2), (dict(sections=(0, 0)), 2), (dict(sections=(3, 3)), 2),
    (dict(sections=(32, 4)), 2), (dict(sections=(2147483647, 2147483647)), 2), (dict(ldx=255), 2), (dict(ldy=248), 2),
    (dict(ldx=260), 2), (dict(x=None), 1), (dict(pos=None), 1), (dict(x=BAD), 3), (dict(y=BAD), 3), (dict(pos=BAD), 3),
    (dict(ldx=320), 1),   # in place with two pitches
])
def test_rope_refusals(L, kw, code):
    assert _rope(L, **kw) == code


def test_rope_empty_batch_is_a_noop(L):
    assert _rope(L, x=None, y=None, pos=None, T=0) == 0


def test_binding_refusals():
    import tensor_transformer_layer_gb300 as mp
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    pos = torch.zeros(1, 4, dtype=torch.int32)
    with pytest.raises(TypeError):
        mp.mp_rope_axes(x.float(), x, pos, sections=(32,))
    with pytest.raises(ValueError):
        mp.mp_rope_axes(x, x, pos, sections=(32,))             # not on the GPU
    with pytest.raises(ValueError):
        mp.mp_rope_axes(x.transpose(0, 1), x, pos, sections=(32,))
    with pytest.raises(ValueError):
        mp.mp_glu_fwd(x[0], x[0], x[0], x[0], x[0], t=1, act="relu")


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device answer")
def test_no_device_answer(L):
    assert _glu(L) == 4
    assert _rope(L) == 4


def _attn(L, nseq=2, Tq=300, Tk=300, max_q=200, max_k=200, heads=4, kv=2, d=64, ld=None, causal=1, scale=0.125, Q=FAKE,
          K=FAKE, O=FAKE, LSE=FAKE, cu=FAKE, st=None):
    ld = ld or {}
    q, k = heads * d, kv * d
    lq, lk = ld.get("q", q), ld.get("k", k)
    fwd = L.mp_attn_varlen_fwd(Q, K, FAKE, O, LSE, cu, FAKE, nseq, Tq, Tk, max_q, max_k, heads, kv, d, lq, lk,
                               ld.get("v", k), ld.get("o", q), causal, scale, st, None)
    bwd = L.mp_attn_varlen_bwd(Q, K, FAKE, O, LSE, FAKE, FAKE, FAKE, FAKE, FAKE, cu, FAKE, nseq, Tq, Tk, max_q, max_k,
                               heads, kv, d, lq, lk, ld.get("v", k), ld.get("o", q), q, q, k, k, causal, scale, st, None)
    assert fwd == bwd
    return fwd


@pytest.mark.parametrize("kw,code", [
    (dict(nseq=-1), 1), (dict(Tq=-1), 1), (dict(Tk=-1), 1), (dict(max_q=-1), 1), (dict(heads=0), 1), (dict(kv=0), 1),
    (dict(d=0), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1),
    (dict(d=80), 2), (dict(heads=3), 2), (dict(max_q=301), 2), (dict(max_k=301), 2), (dict(ld={"q": 255}), 2),
    (dict(ld={"q": 260}), 2), (dict(ld={"k": 120}), 2), (dict(ld={"v": 132}), 2), (dict(ld={"o": 248}), 2),
    (dict(nseq=2147483647, Tq=2147483647, max_q=2147483647), 2), (dict(heads=1 << 24, kv=1 << 24), 2),
    (dict(Q=None), 1), (dict(K=None), 1), (dict(O=None), 1), (dict(LSE=None), 1), (dict(cu=None), 1),
    (dict(Q=BAD), 3), (dict(K=BAD), 3), (dict(O=BAD), 3), (dict(LSE=BAD), 3), (dict(cu=BAD), 3), (dict(st=BAD), 3),
])
def test_attn_varlen_refusals(L, kw, code):
    assert _attn(L, **kw) == code


def test_attn_varlen_no_sequences_is_a_noop(L):
    assert _attn(L, nseq=0, Q=None, cu=None) == 0
    assert _attn(L, max_q=0, max_k=0, Q=None, cu=None) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device answer")
def test_attn_varlen_no_device_answer(L):
    assert _attn(L) == 4


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device answer")
def test_attn_varlen_takes_many_sequences_under_a_long_maximum(L):
    # 4096 sequences of which one may be 131,072 long: the tiles that can exist are few
    kw = dict(nseq=4096, max_q=131072, max_k=131072, heads=64, kv=8)
    assert _attn(L, Tq=1 << 20, Tk=1 << 20, **kw) == 4
    # more tiles than a grid has CTAs
    assert _attn(L, Tq=2147483647, Tk=2147483647, **{**kw, "nseq": 1 << 22}) == 2
    assert _attn(L, Tq=1 << 20, Tk=2147483647, **{**kw, "nseq": 1 << 22, "max_q": 100}) == 2


def test_binding_refuses_numbers_that_a_c_int_would_cut():
    # 2^32 would arrive as 0: a call that does nothing and says that all is well
    import tensor_transformer_layer_gb300 as mp
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    f, cu = torch.zeros(2, 4), torch.tensor([0, 4], dtype=torch.int32)
    for kw in (dict(max_q=1 << 32, max_k=4), dict(max_q=4, max_k=(1 << 32) + 4)):
        with pytest.raises(ValueError, match="32 bits"):
            mp.mp_attn_varlen_fwd(x, x, x, x, f, cu, cu, causal=True, **kw)
        with pytest.raises(ValueError, match="32 bits"):
            mp.mp_attn_varlen_bwd(x, x, x, x, f, x, x, x, x, f, cu, cu, causal=True, **kw)
    with pytest.raises(ValueError, match="32 bits"):
        mp.mp_glu_fwd(x[0], x[0], x[0], x[0], x[0], t=(1 << 32) + 1)
    with pytest.raises(ValueError, match="32 bits"):
        mp.mp_glu_bwd(*[x[0]] * 10, t=(1 << 32) + 1)
    with pytest.raises(ValueError, match="32 bits"):
        mp._int_array(((1 << 32) + 16,))
