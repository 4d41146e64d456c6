"""GPU parity of the packed attention and its gradients against the float64 oracle.

Tolerances (relative Frobenius): each rounding to bf16 on a result's path is off by at most half a step,
2^-8 of the value, independently of the others: sqrt(roundings) * 2^-8. O and dV: the probabilities and
the result. dQ and dK: O (through delta), dS and the result. The log-sum-exp is fp32 throughout: scores
of a few units summed from d <= 128 products, 2^-24 * 128 * 16 < 2e-4 at worst, plus ex2's 2^-22 relative."""
import math

import numpy as np
import pytest
import torch

import oracle
import synth
from gpu_util import f64, mp, rel_fro, status_tensor

pytestmark = pytest.mark.gpu
HALF = 2.0 ** -8
TOL = {"O": math.sqrt(2) * HALF, "dV": math.sqrt(2) * HALF, "dQ": math.sqrt(3) * HALF, "dK": math.sqrt(3) * HALF}
LSE_ABS = 2e-4


def _cu(lens, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(lens)]), dtype=torch.int32)


def _nan(*shape, dtype=torch.bfloat16):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def _inputs(Tq, Tk, heads, kv, d, seed):
    return {"Q": synth.normal_bf16((Tq, heads, d), 1.0, seed), "K": synth.normal_bf16((Tk, kv, d), 1.0, seed + 1),
            "V": synth.normal_bf16((Tk, kv, d), 1.0, seed + 2), "dO": synth.normal_bf16((Tq, heads, d), 1.0, seed + 3)}


def _run(inp, cu_q, cu_k, causal, scale=None, max_q=None, max_k=None, status=0, grad=True):
    dev = {k: v.cuda() for k, v in inp.items()}
    (Tq, heads, d), (Tk, kv, _) = inp["Q"].shape, inp["K"].shape
    cq, ck = cu_q.cuda(), cu_k.cuda()
    kw = dict(max_q=int((cu_q[1:] - cu_q[:-1]).max()) if max_q is None else max_q,
              max_k=int((cu_k[1:] - cu_k[:-1]).max()) if max_k is None else max_k, causal=causal, scale=scale)
    st = status_tensor()
    o = {"O": _nan(Tq, heads, d), "LSE": _nan(heads, Tq, dtype=torch.float32)}
    mp().mp_attn_varlen_fwd(dev["Q"], dev["K"], dev["V"], o["O"], o["LSE"], cq, ck, d_status=st, **kw)
    if grad:
        o.update(dQ=_nan(Tq, heads, d), dK=_nan(Tk, kv, d), dV=_nan(Tk, kv, d))
        delta = _nan(heads, Tq, dtype=torch.float32)
        mp().mp_attn_varlen_bwd(dev["Q"], dev["K"], dev["V"], o["O"], o["LSE"], dev["dO"], o["dQ"], o["dK"], o["dV"],
                                delta, cq, ck, d_status=st, **kw)
    torch.cuda.synchronize()
    assert int(st.item()) == status, int(st.item())
    return {k: v.cpu() for k, v in o.items()}


def _check(got, inp, cu_q, cu_k, causal, scale=None):
    x = {k: f64(v) for k, v in inp.items()}
    scale = inp["Q"].shape[2] ** -0.5 if scale is None else scale
    cq, ck = cu_q.numpy(), cu_k.numpy()
    O, LSE = oracle.attn_varlen_fwd(x["Q"], x["K"], x["V"], cq, ck, causal, scale)
    want = {"O": O}
    if "dQ" in got:
        want.update(oracle.attn_varlen_bwd(x["Q"], x["K"], x["V"], x["dO"], cq, ck, causal, scale))
    lse = got["LSE"].double().numpy()
    assert np.array_equal(np.isneginf(lse), np.isneginf(LSE)) and not np.isnan(lse).any()
    fin = np.isfinite(LSE)
    assert np.all(np.abs(lse[fin] - LSE[fin]) <= LSE_ABS)
    for k, w in want.items():
        g = f64(got[k])
        assert np.isfinite(g).all(), k
        if np.abs(w).max(initial=0.0) == 0.0:
            assert not g.any(), k
        else:
            assert rel_fro(g, w) <= TOL[k], (k, rel_fro(g, w))
    # rows without keys are exactly zero
    dead = np.isneginf(LSE).T
    assert not f64(got["O"])[dead].any()
    if "dQ" in got:
        assert not f64(got["dQ"])[dead].any()


CASES = [
    # q_lens, k_lens (None: the same), heads, kv_heads
    ([2], None, 1, 1),
    ([127, 128, 129], None, 2, 2),
    ([1, 17, 64, 130], None, 4, 4),
    ([256], None, 2, 1),
    ([300, 1, 0, 77, 513], None, 6, 2),
    ([5, 0, 9, 40], [0, 7, 300, 39], 4, 2),        # no keys, no queries, a prefix, a row without keys
    ([140, 260], [3, 129], 3, 1),                  # many rows without keys where causal
    ([33, 200], [400, 641], 5, 5),
    ([1, 1, 1], [129, 1000, 128], 4, 1),           # single queries over long keys
    ([700], [1], 2, 2),                            # one key
]


@pytest.mark.parametrize("q_lens,k_lens,heads,kv", CASES)
@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_attn_varlen_matches_oracle(q_lens, k_lens, heads, kv, d, causal):
    k_lens = q_lens if k_lens is None else k_lens
    cu_q, cu_k = _cu(q_lens), _cu(k_lens)
    inp = _inputs(sum(q_lens), sum(k_lens), heads, kv, d, seed=22000 + sum(q_lens) + d)
    if k_lens == [1]:
        # one key: dS is exactly P (dP - delta) = rounding around 0; only O and dV have a size
        got = _run(inp, cu_q, cu_k, causal)
        x = {k: f64(v) for k, v in inp.items()}
        want = oracle.attn_varlen_bwd(x["Q"], x["K"], x["V"], x["dO"], [0, 700], [0, 1], causal, d ** -0.5)
        assert rel_fro(f64(got["dV"]), want["dV"]) <= TOL["dV"]
        assert np.abs(f64(got["dQ"])).max() <= 1e-3 and np.abs(f64(got["dK"])).max() <= 1e-3 * math.sqrt(700)
        got = {k: got[k] for k in ("O", "LSE")}
    else:
        got = _run(inp, cu_q, cu_k, causal)
    _check(got, inp, cu_q, cu_k, causal)


@pytest.mark.parametrize("d", [64, 96, 128])
def test_attn_varlen_many_tiles(d):
    # more key and query tiles than any ring has stages, shared heads, several waves of work
    lens = [1500, 777, 1024]
    cu = _cu(lens)
    inp = _inputs(sum(lens), sum(lens), 4, 2, d, seed=22500 + d)
    _check(_run(inp, cu, cu, True), inp, cu, cu, True)


@pytest.mark.parametrize("nseq", [32, 33, 71])
@pytest.mark.parametrize("same,causal", [(True, True), (False, True), (False, False)])
def test_attn_varlen_many_sequences(nseq, same, causal):
    # more sequences than a warp has lanes, of all lengths from none to several tiles, the longest among the last
    rng = np.random.default_rng(22550 + nseq)
    q_lens = rng.choice([0, 1, 31, 128, 129, 200], nseq)
    k_lens = q_lens if same else rng.choice([0, 1, 40, 128, 300], nseq)
    q_lens[-2] = 600
    k_lens[-2] = 600
    cu_q, cu_k = _cu(q_lens), _cu(k_lens)
    inp = _inputs(int(sum(q_lens)), int(sum(k_lens)), 2, 1, 64, seed=22560 + nseq)
    _check(_run(inp, cu_q, cu_k, causal), inp, cu_q, cu_k, causal)


@pytest.mark.parametrize("q_lens,k_lens,heads,kv", [
    ([1], [9000], 4, 1),                       # clusters of eight CTAs share a query's keys
    ([1, 3, 2], [2100, 4097, 1], 2, 2),
    ([130, 1], [4000, 3900], 3, 1),            # of four; a second query tile of two rows
    ([1100], [1100], 2, 1),                    # causal: parts that some rows see nothing of
    ([900], [1500], 1, 1),
    ([2300, 40], [2200, 900], 2, 2),           # rows without keys where causal
])
@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_attn_varlen_long_keys_for_few_queries(q_lens, k_lens, heads, kv, d, causal):
    cu_q, cu_k = _cu(q_lens), _cu(k_lens)
    inp = _inputs(sum(q_lens), sum(k_lens), heads, kv, d, seed=22700 + sum(q_lens) + d)
    _check(_run(inp, cu_q, cu_k, causal), inp, cu_q, cu_k, causal)


def test_attn_varlen_scale_and_large_scores():
    # scores up to +-200 and a jump of the running maximum at every key tile
    lens = [400]
    cu = _cu(lens)
    inp = _inputs(400, 400, 2, 2, 64, seed=22600)
    inp["K"] = (inp["K"].float() * torch.linspace(0.1, 6, 400)[:, None, None]).to(torch.bfloat16)
    for causal in (True, False):
        got = _run(inp, cu, cu, causal, scale=0.5, grad=False)
        _check(got, inp, cu, cu, causal, scale=0.5)


def test_attn_varlen_other_sequences_do_not_leak():
    # the second sequence is all NaN, the third infinite: neither reaches the first, nor the rows behind
    lens = [200, 150, 33]
    cu = _cu(lens)
    clean = _inputs(sum(lens), sum(lens), 2, 1, 96, seed=22700)
    dirty = {k: v.clone() for k, v in clean.items()}
    for v in dirty.values():
        v[200:350] = float("nan")
        v[350:] = float("inf")
    for causal in (True, False):
        a, b = _run(clean, cu, cu, causal), _run(dirty, cu, cu, causal)
        for k in a:
            sl = (slice(None), slice(0, 200)) if k == "LSE" else slice(0, 200)
            assert torch.equal(a[k][sl], b[k][sl]), (k, causal)


def test_attn_varlen_rows_outside_sequences_stay():
    # 10 rows before the first sequence and 20 behind the last are not written
    cu = _cu([100, 60], first=10)
    inp = _inputs(190, 190, 2, 2, 64, seed=22800)
    got = _run(inp, cu, cu, True)
    for k in ("O", "dQ", "dK", "dV"):
        assert torch.isnan(got[k][:10].float()).all() and torch.isnan(got[k][170:].float()).all(), k
        assert torch.isfinite(got[k][10:170].float()).all(), k
    assert torch.isnan(got["LSE"][:, :10]).all() and torch.isnan(got["LSE"][:, 170:]).all()


def test_attn_varlen_strided_views():
    # the parts of a packed projection and of its gradient, against contiguous copies
    T, heads, kv, d = 333, 4, 2, 64
    cu = _cu([133, 200])
    qkv = synth.normal_bf16((T, heads + 2 * kv, d), 1.0, 22900)
    dO = synth.normal_bf16((T, heads, d), 1.0, 22901)
    inp = {"Q": qkv[:, :heads], "K": qkv[:, heads:heads + kv], "V": qkv[:, heads + kv:], "dO": dO}
    want = _run({k: v.contiguous() for k, v in inp.items()}, cu, cu, True)
    x = qkv.cuda()
    g = torch.full_like(x, 7.0)
    wide = torch.full((T, heads + 3, d), 5.0, dtype=torch.bfloat16, device="cuda")
    O, lse, delta = wide[:, 1:1 + heads], _nan(heads, T, dtype=torch.float32), _nan(heads, T, dtype=torch.float32)
    c = cu.cuda()
    kw = dict(max_q=200, max_k=T, causal=True)   # maxima may be larger than the longest sequence
    q, k, v = x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:]
    mp().mp_attn_varlen_fwd(q, k, v, O, lse, c, c, **kw)
    mp().mp_attn_varlen_bwd(q, k, v, O, lse, dO.cuda(), g[:, :heads], g[:, heads:heads + kv], g[:, heads + kv:], delta, c,
                            c, **kw)
    torch.cuda.synchronize()
    assert torch.equal(O.cpu(), want["O"]) and torch.equal(lse.cpu(), want["LSE"])
    assert torch.all(wide[:, 0] == 5.0) and torch.all(wide[:, 1 + heads:] == 5.0)
    for name, part in (("dQ", g[:, :heads]), ("dK", g[:, heads:heads + kv]), ("dV", g[:, heads + kv:])):
        assert torch.equal(part.cpu(), want[name]), name
    # delta is the definition's sum, within O's rounding of it
    exact = oracle.attn_varlen_fwd(f64(q.cpu()), f64(k.cpu()), f64(v.cpu()), cu.numpy(), cu.numpy(), True, d ** -0.5)[0]
    size = (np.abs(f64(dO)) * np.abs(exact)).sum(-1).T
    assert np.all(np.abs(delta.cpu().numpy() - (f64(dO) * exact).sum(-1).T) <= HALF * size + 1e-4)


def test_attn_varlen_bad_offsets_are_reported_and_left_out():
    # the bad sequence's rows are not touched, the others are right
    inp = _inputs(300, 300, 2, 2, 64, seed=23000)
    good = _cu([100, 100, 100])
    want = _run(inp, good, good, True)
    for cu in ([0, 100, 200, 301], [0, 100, 90, 90], [0, 100, 250, 300]):  # beyond the end, descending, too long
        cu = torch.tensor(cu, dtype=torch.int32)
        got = _run(inp, cu, cu, True, max_q=100, max_k=100, status=mp().MP_DEV_SEQ_RANGE)
        for k in ("O", "dQ", "dK", "dV"):
            assert torch.equal(got[k][:100], want[k][:100]), k
            assert torch.isnan(got[k][200:250].float()).all(), k
    assert mp().mp_status_from_device(mp().MP_DEV_SEQ_RANGE) == 9


def test_attn_varlen_repeats_exactly_and_in_a_graph():
    lens = [513, 40, 300]
    cu = _cu(lens)
    T = sum(lens)
    inp = _inputs(T, T, 4, 2, 128, seed=23100)
    want = _run(inp, cu, cu, True)
    for _ in range(5):
        got = _run(inp, cu, cu, True)
        for k in want:
            assert torch.equal(got[k], want[k]), k
    dev = {k: v.cuda() for k, v in inp.items()}
    o = {"O": _nan(T, 4, 128), "LSE": _nan(4, T, dtype=torch.float32), "dQ": _nan(T, 4, 128), "dK": _nan(T, 2, 128),
         "dV": _nan(T, 2, 128)}
    delta, c = _nan(4, T, dtype=torch.float32), cu.cuda()
    kw = dict(max_q=513, max_k=513, causal=True)

    def step():
        mp().mp_attn_varlen_fwd(dev["Q"], dev["K"], dev["V"], o["O"], o["LSE"], c, c, **kw)
        mp().mp_attn_varlen_bwd(dev["Q"], dev["K"], dev["V"], o["O"], o["LSE"], dev["dO"], o["dQ"], o["dK"], o["dV"],
                                delta, c, c, **kw)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step()
    for v in o.values():
        v.fill_(float("nan"))
    g.replay()
    torch.cuda.synchronize()
    for k in o:
        assert torch.equal(o[k].cpu(), want[k]), k


def test_attn_varlen_nothing_to_do():
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    f = torch.empty(2, 0, dtype=torch.float32, device="cuda")
    cu0 = torch.zeros(3, dtype=torch.int32, device="cuda")
    mp().mp_attn_varlen_fwd(e, e, e, e, f, cu0, cu0, max_q=0, max_k=0, causal=True)
    mp().mp_attn_varlen_bwd(e, e, e, e, f, e, e, e, e, f, cu0, cu0, max_q=0, max_k=0, causal=True)
    # queries without any key in the whole batch; keys without any query
    q = synth.normal_bf16((5, 2, 64), 1.0, 23200).cuda()
    O, dQ, lse, dl = _nan(5, 2, 64), _nan(5, 2, 64), _nan(2, 5, dtype=torch.float32), _nan(2, 5, dtype=torch.float32)
    cq = torch.tensor([0, 2, 5], dtype=torch.int32, device="cuda")
    mp().mp_attn_varlen_fwd(q, e, e, O, lse, cq, cu0, max_q=3, max_k=0, causal=False)
    mp().mp_attn_varlen_bwd(q, e, e, O, lse, q, dQ, e, e, dl, cq, cu0, max_q=3, max_k=0, causal=False)
    dK, dV = _nan(5, 2, 64), _nan(5, 2, 64)
    mp().mp_attn_varlen_bwd(e, q, q, e, f, e, e, dK, dV, f, cu0, cq, max_q=0, max_k=3, causal=True)
    torch.cuda.synchronize()
    for x in (O, dQ, dK, dV):
        assert torch.all(x == 0)
    assert torch.isneginf(lse).all()


def test_attn_varlen_zero_wait_budget(monkeypatch):
    # The kernels' waits are short: a budget of zero may or may not run out. Each call ends either way, says
    # so where it did, is right where it did not, and the context stays usable.
    lens = [1024]
    cu = _cu(lens)
    inp = _inputs(1024, 1024, 2, 2, 64, seed=23300)
    want = _run(inp, cu, cu, True)
    monkeypatch.setenv("MPTP_WAIT_BUDGET_NS", "0")
    dev = {k: v.cuda() for k, v in inp.items()}
    c = cu.cuda()
    st = status_tensor()
    o, lse, dl = _nan(1024, 2, 64), _nan(2, 1024, dtype=torch.float32), _nan(2, 1024, dtype=torch.float32)
    g = [_nan(1024, 2, 64) for _ in range(3)]
    kw = dict(max_q=1024, max_k=1024, causal=True, d_status=st)
    mp().mp_attn_varlen_fwd(dev["Q"], dev["K"], dev["V"], o, lse, c, c, **kw)
    torch.cuda.synchronize()
    assert int(st.item()) == mp().MP_DEV_TIMEOUT or torch.equal(o.cpu(), want["O"])
    st.zero_()
    mp().mp_attn_varlen_bwd(dev["Q"], dev["K"], dev["V"], want["O"].cuda(), want["LSE"].cuda(), dev["dO"], *g, dl, c, c,
                            **kw)
    torch.cuda.synchronize()
    assert int(st.item()) == mp().MP_DEV_TIMEOUT or all(torch.equal(a.cpu(), want[k])
                                                        for a, k in zip(g, ("dQ", "dK", "dV")))
    monkeypatch.delenv("MPTP_WAIT_BUDGET_NS")
    got = _run(inp, cu, cu, True)
    for k in want:
        assert torch.equal(got[k], want[k]), k


@pytest.mark.parametrize("lens,heads,kv", [
    ([600], 4, 2),            # two CTAs a key tile
    ([1000], 2, 1),           # four
    ([1000], 8, 1),           # eight
    ([130, 900, 5], 6, 1),    # parts that end inside a head; sequences with fewer iterations than CTAs
])
@pytest.mark.parametrize("d", [64, 96, 128])
def test_attn_varlen_shared_key_tiles(lens, heads, kv, d):
    # few key tiles with many queries each: clusters of CTAs share a tile and join their sums
    cu = _cu(lens)
    inp = _inputs(sum(lens), sum(lens), heads, kv, d, seed=23400 + heads + d)
    for causal in (True, False):
        got = _run(inp, cu, cu, causal)
        _check(got, inp, cu, cu, causal)
        again = _run(inp, cu, cu, causal)
        for k in got:
            assert torch.equal(got[k], again[k]), k


@pytest.mark.parametrize("same", [True, False])
def test_attn_varlen_a_thousand_sequences(same):
    # most of a token or two, or empty; a long one among the last
    rng = np.random.default_rng(23500)
    q_lens = rng.choice([0, 1, 1, 2, 3, 17], 1100)
    k_lens = q_lens if same else rng.choice([0, 1, 2, 5, 40], 1100)
    q_lens[1090] = k_lens[1090] = 700
    cu_q, cu_k = _cu(q_lens), _cu(k_lens)
    inp = _inputs(int(sum(q_lens)), int(sum(k_lens)), 2, 1, 64, seed=23510)
    got = _run(inp, cu_q, cu_k, True, max_q=700, max_k=int(sum(k_lens)))
    _check(got, inp, cu_q, cu_k, True)


def test_attn_varlen_a_bad_sequence_far_back_is_reported():
    # the sequence behind a thousand others is too long: the call says so, and the others are right
    lens = [3] * 1000 + [50]
    cu = _cu(lens)
    inp = _inputs(sum(lens), sum(lens), 2, 2, 64, seed=23600)
    want = _run(inp, cu, cu, True)
    got = _run(inp, cu, cu, True, max_q=40, max_k=40, status=mp().MP_DEV_SEQ_RANGE)
    for k in ("O", "dQ", "dK", "dV"):
        assert torch.equal(got[k][:3000], want[k][:3000]) and torch.isnan(got[k][3000:].float()).all(), k
