"""GPU parity of the gated feed-forward block against the float64 oracle.

Tolerances (relative Frobenius): each rounding to bf16 on a result's path is off by at most half a step,
2^-8 of the value, independently of the others: sqrt(roundings) * 2^-8. Y: itself. Z: Y, Z. dWd: Y, dWd.
GU: itself. dGU: GU, dGU. dX and dW: GU, dGU, and the result."""
import math

import numpy as np
import pytest
import torch

import oracle
import synth
from gpu_util import f64, mp, rel_fro, status_tensor

pytestmark = pytest.mark.gpu
HALF = 2.0 ** -8
TOL = {"Y": HALF, "Z": math.sqrt(2) * HALF, "GU": HALF, "dGU": math.sqrt(2) * HALF, "dX": math.sqrt(3) * HALF,
       "dW": math.sqrt(3) * HALF, "dWd": math.sqrt(2) * HALF}


def _inputs(T, h, f, seed):
    return {"X": synth.normal_bf16((T, h), 1.0, seed), "W": synth.normal_bf16((h, 2 * f), 1.0 / math.sqrt(h), seed + 1),
            "Wd": synth.normal_bf16((f, h), 1.0 / math.sqrt(f), seed + 2), "dZ": synth.normal_bf16((T, h), 1.0, seed + 3)}


def _nan(*shape):
    return torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")


def _run(inp, t, act, save=True):
    d = {k: v.cuda() for k, v in inp.items()}
    T, h = inp["X"].shape
    f = inp["Wd"].shape[0]
    o = {"Z": _nan(T, h), "Y": _nan(T, f), "GU": _nan(T, 2 * f) if save else None}
    st = status_tensor()
    mp().mp_glu_fwd(d["X"], d["W"], d["Wd"], o["Z"], o["Y"], o["GU"], t=t, act=act, d_status=st)
    if save:
        o.update(dX=_nan(T, h), dW=_nan(h, 2 * f), dWd=_nan(f, h), dGU=_nan(T, 2 * f))
        mp().mp_glu_bwd(d["X"], d["W"], d["Wd"], o["GU"], o["Y"], d["dZ"], o["dX"], o["dW"], o["dWd"], o["dGU"], t=t,
                        act=act, d_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    return o


@pytest.mark.parametrize("T,h,f,t", [
    (1, 64, 64, 1),          # the least of everything
    (1, 1536, 1024, 8),      # one token
    (2, 256, 320, 1),        # an odd number of 64-wide blocks
    (7, 128, 192, 3),
    (16, 512, 512, 2),
    (65, 320, 448, 1),
    (127, 192, 1024, 4),
    (129, 128, 256, 2),
    (256, 256, 640, 2),
    (257, 704, 576, 1),
    (300, 256, 1024, 4),
    (1000, 384, 192, 1),
])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_glu_matches_oracle(T, h, f, t, act):
    inp = _inputs(T, h, f, seed=21000 + T + h)
    got = _run(inp, t, act)
    x = {k: f64(v) for k, v in inp.items()}
    want = dict(zip(("GU", "Y", "Z"), oracle.glu_fwd(x["X"], x["W"], x["Wd"], act)))
    want.update(oracle.glu_bwd(x["X"], x["W"], x["Wd"], x["dZ"], act))
    errs = {k: rel_fro(f64(got[k].cpu()), want[k]) for k in want}
    assert all(errs[k] <= TOL[k] for k in errs), errs
    # the forward gives the same Y and Z whether gate and up are kept or not
    lean = _run(inp, t, act, save=False)
    assert torch.equal(lean["Y"], got["Y"]) and torch.equal(lean["Z"], got["Z"])


@pytest.mark.parametrize("T,h,f,t", [
    (128, 256, 320, 1),      # two slices of 64 for the gated product, one of 128 for the other
    (130, 1536, 4096, 4),    # two: 80 and 50 tokens, each over several CTAs of a cluster
    (159, 64, 64, 1),
    (161, 320, 192, 1),      # 96 and 65
    (241, 704, 1024, 2),     # 128 and 113
    (255, 448, 576, 1),
])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_glu_matches_oracle_where_the_tokens_are_cut(T, h, f, t, act):
    test_glu_matches_oracle(T, h, f, t, act)


@pytest.mark.parametrize("T,h,f,t", [
    (257, 704, 6592, 1),     # large tiles: too many blocks of columns for three slices; an odd number of 64
    (1000, 384, 2496, 3),
    (1300, 192, 2048, 4),
    (2500, 320, 1024, 1),
    (20000, 64, 64, 1),
])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_glu_matches_oracle_on_large_tiles(T, h, f, t, act):
    test_glu_matches_oracle(T, h, f, t, act)


@pytest.mark.parametrize("T,h,f", [
    (400, 64, 64),           # one tile a launch: its loads behind the last column are zero fills
    (400, 64, 128),
    (400, 64, 192),
    (2600, 128, 2112),       # 99 tiles, more than CTA pairs: a pair's second tile follows one that ends early
    (2600, 128, 2176),
    (2600, 128, 2240),
])
def test_glu_gradients_where_columns_end_inside_a_tile(T, h, f):
    # Large tiles are 256 columns wide; the gradients' boxes of the last columns are stored before they are loaded again.
    inp = _inputs(T, h, f, seed=21170)
    first = _run(inp, 1, "silu")
    x = {k: f64(v) for k, v in inp.items()}
    want = oracle.glu_bwd(x["X"], x["W"], x["Wd"], x["dZ"], "silu")
    errs = {k: rel_fro(f64(first[k].cpu()), want[k]) for k in want}
    assert all(errs[k] <= TOL[k] for k in errs), errs
    d = {k: v.cuda() for k, v in inp.items()}
    for _ in range(20):
        o = {"dX": _nan(T, h), "dW": _nan(h, 2 * f), "dWd": _nan(f, h), "dGU": _nan(T, 2 * f)}
        mp().mp_glu_bwd(d["X"], d["W"], d["Wd"], first["GU"], first["Y"], d["dZ"], o["dX"], o["dW"], o["dWd"], o["dGU"],
                        t=1, act="silu")
        for k in o:
            assert torch.equal(o[k], first[k]), k


def test_glu_large_tiles_do_not_depend_on_shards():
    inp = _inputs(2600, 256, 1024, seed=21150)
    ref = _run(inp, 1, "silu")
    for t in (2, 4, 8):
        got = _run(inp, t, "silu")
        for k in ref:
            assert torch.equal(got[k], ref[k]), (t, k)


def test_glu_does_not_depend_on_shards_and_repeats_exactly():
    inp = _inputs(300, 256, 1024, seed=21100)
    ref = _run(inp, 1, "silu")
    for t in (1, 2, 4, 8):
        got = _run(inp, t, "silu")
        for k in ref:
            assert torch.equal(got[k], ref[k]), (t, k)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_glu_extreme_gates(act):
    # gates far out on both sides: act is 0 or the gate itself, its slope 0 or 1, and nothing is NaN
    T, h, f = 64, 64, 128
    inp = _inputs(T, h, f, seed=21200)
    inp["X"] = torch.zeros_like(inp["X"])
    inp["X"][:, 0] = torch.linspace(-1, 1, T).to(torch.bfloat16)
    inp["W"][0, :f] = 20000.0
    inp["W"][0, f:] = 1.0
    got = _run(inp, 2, act)
    x = {k: f64(v) for k, v in inp.items()}
    want = dict(zip(("GU", "Y", "Z"), oracle.glu_fwd(x["X"], x["W"], x["Wd"], act)))
    want.update(oracle.glu_bwd(x["X"], x["W"], x["Wd"], x["dZ"], act))
    errs = {k: rel_fro(f64(got[k].cpu()), want[k]) for k in want}
    assert all(errs[k] <= TOL[k] for k in errs), errs


def test_glu_empty_batch():
    h, f = 64, 128
    W, Wd = _nan(h, 2 * f), _nan(f, h)
    e = torch.empty(0, h, dtype=torch.bfloat16, device="cuda")
    ef, e2 = (torch.empty(0, n, dtype=torch.bfloat16, device="cuda") for n in (f, 2 * f))
    mp().mp_glu_fwd(e, W, Wd, e, ef, e2, t=1)
    dW, dWd = _nan(h, 2 * f), _nan(f, h)
    mp().mp_glu_bwd(e, W, Wd, e2, ef, e, e, dW, dWd, e2, t=1)
    assert torch.all(dW == 0) and torch.all(dWd == 0)


def test_glu_graph_capture_and_other_stream():
    inp = _inputs(200, 256, 512, seed=21300)
    want = _run(inp, 2, "silu")
    d = {k: v.cuda() for k, v in inp.items()}
    T, h, f = 200, 256, 512
    o = {"Z": _nan(T, h), "Y": _nan(T, f), "GU": _nan(T, 2 * f), "dX": _nan(T, h), "dW": _nan(h, 2 * f),
         "dWd": _nan(f, h), "dGU": _nan(T, 2 * f)}

    def step():
        mp().mp_glu_fwd(d["X"], d["W"], d["Wd"], o["Z"], o["Y"], o["GU"], t=2)
        mp().mp_glu_bwd(d["X"], d["W"], d["Wd"], o["GU"], o["Y"], d["dZ"], o["dX"], o["dW"], o["dWd"], o["dGU"], t=2)

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
        assert torch.equal(o[k], want[k]), k


def test_glu_wait_budget_exhaustion(monkeypatch):
    inp = _inputs(256, 4096, 512, seed=21400)
    d = {k: v.cuda() for k, v in inp.items()}
    Z, Y = _nan(256, 4096), _nan(256, 512)
    st = status_tensor()
    monkeypatch.setenv("MPTP_WAIT_BUDGET_NS", "0")
    mp().mp_glu_fwd(d["X"], d["W"], d["Wd"], Z, Y, None, t=1, d_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) & mp().MP_DEV_TIMEOUT
    monkeypatch.delenv("MPTP_WAIT_BUDGET_NS")
    got = _run(inp, 1, "silu", save=False)
    want = oracle.glu_fwd(*(f64(inp[k]) for k in ("X", "W", "Wd")), "silu")
    assert rel_fro(f64(got["Z"].cpu()), want[2]) <= TOL["Z"]


def test_glu_wait_budget_exhaustion_on_large_tiles(monkeypatch):
    inp = _inputs(2600, 2048, 1024, seed=21500)
    d = {k: v.cuda() for k, v in inp.items()}
    Z, Y = _nan(2600, 2048), _nan(2600, 1024)
    st = status_tensor()
    monkeypatch.setenv("MPTP_WAIT_BUDGET_NS", "0")
    mp().mp_glu_fwd(d["X"], d["W"], d["Wd"], Z, Y, None, t=1, d_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) & mp().MP_DEV_TIMEOUT
    monkeypatch.delenv("MPTP_WAIT_BUDGET_NS")
    got = _run(inp, 1, "silu", save=False)
    want = oracle.glu_fwd(*(f64(inp[k]) for k in ("X", "W", "Wd")), "silu")
    assert rel_fro(f64(got["Z"].cpu()), want[2]) <= TOL["Z"]


def test_glu_bwd_wait_budget_exhaustion_with_few_tokens(monkeypatch):
    inp = _inputs(64, 4096, 512, seed=21600)
    good = _run(inp, 1, "silu")
    d = {k: v.cuda() for k, v in inp.items()}
    o = {"dX": _nan(64, 4096), "dW": _nan(4096, 1024), "dWd": _nan(512, 4096), "dGU": _nan(64, 1024)}
    st = status_tensor()
    monkeypatch.setenv("MPTP_WAIT_BUDGET_NS", "0")
    mp().mp_glu_bwd(d["X"], d["W"], d["Wd"], good["GU"], good["Y"], d["dZ"], o["dX"], o["dW"], o["dWd"], o["dGU"], t=1,
                    act="silu", d_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) & mp().MP_DEV_TIMEOUT
    monkeypatch.delenv("MPTP_WAIT_BUDGET_NS")
    again = _run(inp, 1, "silu")
    for k in good:
        assert torch.equal(again[k], good[k]), k


@pytest.mark.parametrize("T,h,f", [(9, 1536, 4096), (64, 512, 2048), (1, 64, 64)])
def test_glu_with_few_tokens_stores_nothing_without_a_part(T, h, f, monkeypatch):
    # Under a wait budget of zero the last CTA of every cluster (or each CTA alone) has no loads: no CTA of it stores.
    inp = _inputs(T, h, f, seed=21700)
    good = _run(inp, 1, "silu")
    d = {k: v.cuda() for k, v in inp.items()}
    o = {"Z": _nan(T, h), "Y": _nan(T, f), "GU": _nan(T, 2 * f), "dX": _nan(T, h), "dGU": _nan(T, 2 * f)}
    dW, dWd = _nan(h, 2 * f), _nan(f, h)
    monkeypatch.setenv("MPTP_WAIT_BUDGET_NS", "0")
    mp().mp_glu_fwd(d["X"], d["W"], d["Wd"], o["Z"], o["Y"], o["GU"], t=1, act="silu")
    mp().mp_glu_bwd(d["X"], d["W"], d["Wd"], good["GU"], good["Y"], d["dZ"], o["dX"], dW, dWd, o["dGU"], t=1, act="silu")
    torch.cuda.synchronize()
    for k, v in o.items():
        assert torch.isnan(v.float()).all(), k
    monkeypatch.delenv("MPTP_WAIT_BUDGET_NS")
    again = _run(inp, 1, "silu")
    for k in good:
        assert torch.equal(again[k], good[k]), k
