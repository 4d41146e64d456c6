"""GPU parity of the norm of queries and keys with the rotation, and of its gradients, against the float64 oracle.

Tolerances per element. A result in bf16 is off by half a step, 2^-8 of it. Before that: the angle (within 2^-20 turns,
6e-6 radians) on a pair's two elements, and fp32 arithmetic, a handful of roundings of 2^-24 and rsqrt's 2^-22: 1e-5 of
the pair's magnitudes for y, twice that for dx (g through the angle once more in the mean). dw is fp32: 1e-5 of each
addend, and 2^-24 of the sum of magnitudes for each addition in a row (at most 100 in these sizes): 2e-5 of them."""
import numpy as np
import pytest
import torch

import oracle
import synth
from gpu_util import f64, mp

pytestmark = pytest.mark.gpu
EPS = 1e-6


def _pairs(a, sections, interleaved):
    """|a| + |b| of each element's pair (an element outside every pair: its own magnitude)."""
    n, size = sum(sections), np.abs(a)
    if interleaved:
        both = size[..., 0:2 * n:2] + size[..., 1:2 * n:2]
        size[..., 0:2 * n:2] = size[..., 1:2 * n:2] = both
    else:
        size[..., :n] = size[..., n:2 * n] = size[..., :n] + size[..., n:2 * n]
    return size


def _inputs(T, heads, d, axes, top, seed):
    g = torch.Generator().manual_seed(seed)
    x = synth.normal_bf16((T, heads, d), 1.0, seed + 1)
    x = (x.float() * torch.exp(torch.randn(T, heads, 1, generator=g))).to(torch.bfloat16)
    return {"x": x, "dy": synth.normal_bf16((T, heads, d), 1.0, seed + 2),
            "wq": (1 + 0.2 * torch.randn(d, generator=g)).to(torch.bfloat16),
            "wk": (1 + 0.2 * torch.randn(d, generator=g)).to(torch.bfloat16),
            "pos": torch.randint(0, top, (axes, T), generator=g, dtype=torch.int64).to(torch.int32)}


def _nan(*shape, dtype=torch.bfloat16):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def _run(inp, nq, **kw):
    dev = {k: v.cuda() for k, v in inp.items()}
    T, heads, d = inp["x"].shape
    y, dx = _nan(T, heads, d), _nan(T, heads, d)
    dwq, dwk = _nan(d, dtype=torch.float32), _nan(d, dtype=torch.float32)
    ws = _nan(max(1, mp().mp_qk_norm_rope_bwd_workspace_bytes(T, heads, d) // 4), dtype=torch.float32)
    wq, wk = dev["wq"] if nq > 0 else None, dev["wk"] if nq < heads else None
    mp().mp_qk_norm_rope(dev["x"], y, wq, wk, dev["pos"], q_heads=nq, eps=EPS, **kw)
    mp().mp_qk_norm_rope_bwd(dev["x"], dev["dy"], dx, wq, wk, dwq if nq > 0 else None, dwk if nq < heads else None,
                             dev["pos"], ws, q_heads=nq, eps=EPS, **kw)
    return {"y": y.cpu(), "dx": dx.cpu(), "dwq": dwq.cpu(), "dwk": dwk.cpu()}


def _check(got, inp, nq, sections, base=10000.0, interleaved=False, per_axis=False):
    x, dy, wq, wk, pos = f64(inp["x"]), f64(inp["dy"]), f64(inp["wq"]), f64(inp["wk"]), inp["pos"].numpy()
    how = (pos, nq, sections, base, EPS, interleaved, per_axis)
    heads = x.shape[1]
    n = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + EPS)
    w = np.stack([wq if h < nq else wk for h in range(heads)])
    y = oracle.qk_norm_rope(x, wq, wk, *how)
    err = np.abs(f64(got["y"]) - y) - 2.0 ** -8 * np.abs(y) - 1e-5 * _pairs(n * w, sections, interleaved)
    assert np.all(err <= 0), float(err.max())
    want = oracle.qk_norm_rope_bwd(x, dy, wq, wk, *how)
    g = _pairs(dy.copy(), sections, interleaved)
    r = 1.0 / np.sqrt(np.mean(x * x, -1, keepdims=True) + EPS)
    size = r * (np.abs(w) * g + np.abs(n) * np.mean(np.abs(w * n) * g, -1, keepdims=True))
    err = np.abs(f64(got["dx"]) - want["dx"]) - 2.0 ** -8 * np.abs(want["dx"]) - 2e-5 * size
    assert np.all(err <= 0), float(err.max())
    terms = (g * np.abs(n)).sum(0)
    for name, part in (("dwq", terms[:nq].sum(0)), ("dwk", terms[nq:].sum(0))):
        if part.ndim and np.any(part):
            err = np.abs(f64(got[name]) - want[name]) - 2e-5 * part
            assert np.all(err <= 0), (name, float(err.max()))


@pytest.mark.parametrize("T,heads,nq,d,sections,top", [
    (1, 1, 1, 8, (4,), 100),                  # one token, one head, one group of pairs
    (5, 20, 16, 96, (48,), 1 << 20),          # a decoding step: six lanes a head
    (33, 5, 4, 72, (0, 18, 18), 300),         # nine lanes a head, an axis without pairs
    (33, 12, 8, 72, (16, 16), 300),           # eight elements of each head stay unrotated
    (64, 3, 2, 80, (20, 9, 3), 5000),         # sixteen of them
    (257, 9, 8, 128, (64,), 40000),           # one key head
    (19, 3, 1, 256, (32, 32, 32, 32), 999),   # four axes, the widest head
    (7, 2, 1, 256, (64, 60), 2147483647),     # the widest head in narrow vectors, the farthest positions
    (21, 3, 2, 200, (100,), 64),              # 25 lanes a head, one head a warp
    (9, 70, 1, 16, (1, 2, 1), 64),            # many heads of few elements
    (40, 4, 0, 64, (32,), 50),                # keys only
    (40, 4, 4, 64, (8,), 50),                 # queries only, most of a head unrotated
    (3001, 2, 1, 64, (32,), 3000),            # more tokens than warps
])
@pytest.mark.parametrize("interleaved,per_axis", [(False, False), (True, True)])
def test_norm_and_gradients_match_oracle(T, heads, nq, d, sections, top, interleaved, per_axis):
    inp = _inputs(T, heads, d, len(sections), top, 21000 + T + d)
    kw = dict(sections=sections, base=10000.0, interleaved=interleaved, per_axis=per_axis)
    _check(_run(inp, nq, **kw), inp, nq, **kw)


@pytest.mark.parametrize("T,heads,nq,d", [
    (9, 8, 4, 64),        # both kinds in a warp, lanes halved
    (9, 9, 7, 64),        # the last query lane has one head less
    (2600, 10, 5, 96),    # five lanes for five and five heads: apart, a step each
    (1300, 5, 4, 96),     # one step of both
    (70, 7, 1, 128),      # one query head, six key heads
    (1250, 40, 32, 128),  # apart, more blocks than the chip holds
    (2500, 4, 2, 256),    # two lanes' width
    (11, 3, 2, 176),      # two heads at once, eleven lanes each
])
def test_query_and_key_heads_dealt_to_warps(T, heads, nq, d):
    inp = _inputs(T, heads, d, 2, 5000, 21700 + T + d)
    kw = dict(sections=(d // 4, d // 4), base=10000.0, interleaved=T % 2 == 0, per_axis=False)
    _check(_run(inp, nq, **kw), inp, nq, **kw)


def test_strided_rows_and_in_place():
    inp = _inputs(77, 6, 64, 3, 1000, 21500)
    sec = (8, 12, 12)
    want = _run(inp, 4, sections=sec)
    _check(want, inp, 4, sec)
    rows = torch.full((77, 9, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    grads = rows.clone()
    wq, wk, pos = inp["wq"].cuda(), inp["wk"].cuda(), inp["pos"].cuda()
    rows[:, 1:7], grads[:, 2:8] = inp["x"].cuda(), inp["dy"].cuda()
    dwq, dwk = _nan(64, dtype=torch.float32), _nan(64, dtype=torch.float32)
    ws = torch.empty(mp().mp_qk_norm_rope_bwd_workspace_bytes(77, 6, 64), dtype=torch.uint8, device="cuda")
    mp().mp_qk_norm_rope_bwd(rows[:, 1:7], grads[:, 2:8], grads[:, 2:8], wq, wk, dwq, dwk, pos, ws, q_heads=4, sections=sec)
    mp().mp_qk_norm_rope(rows[:, 1:7], rows[:, 1:7], wq, wk, pos, q_heads=4, sections=sec)
    assert torch.equal(rows[:, 1:7].cpu(), want["y"]) and torch.equal(grads[:, 2:8].cpu(), want["dx"])
    assert torch.equal(dwq.cpu(), want["dwq"]) and torch.equal(dwk.cpu(), want["dwk"])
    for t, live in ((rows, slice(1, 7)), (grads, slice(2, 8))):
        rest = t.clone()
        rest[:, live] = 3.0
        assert torch.all(rest == 3.0)


def test_zero_heads_and_no_tokens():
    inp = _inputs(6, 3, 64, 1, 10, 21600)
    inp["x"][2] = 0
    got = _run(inp, 2, sections=(32,))
    assert not got["y"][2].any()
    _check(got, inp, 2, (32,))
    empty = torch.empty(0, 3, 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.empty(1, 0, dtype=torch.int32, device="cuda")
    w, ws = inp["wq"].cuda(), torch.empty(0, dtype=torch.uint8, device="cuda")
    dwq, dwk = _nan(64, dtype=torch.float32), _nan(64, dtype=torch.float32)
    mp().mp_qk_norm_rope(empty, empty, w, w, pos, q_heads=2, sections=(32,))
    mp().mp_qk_norm_rope_bwd(empty, empty, empty, w, w, dwq, dwk, pos, ws, q_heads=2, sections=(32,))
    assert not dwq.any() and not dwk.any()


def test_other_stream_and_replayed_graph():
    inp = _inputs(50, 4, 96, 1, 1000, 21700)
    want = _run(inp, 3, sections=(48,))
    dev = {k: v.cuda() for k, v in inp.items()}
    y, dx = _nan(50, 4, 96), _nan(50, 4, 96)
    dwq, dwk = _nan(96, dtype=torch.float32), _nan(96, dtype=torch.float32)
    ws = torch.empty(mp().mp_qk_norm_rope_bwd_workspace_bytes(50, 4, 96), dtype=torch.uint8, device="cuda")

    def step(**kw):
        mp().mp_qk_norm_rope(dev["x"], y, dev["wq"], dev["wk"], dev["pos"], q_heads=3, sections=(48,), **kw)
        mp().mp_qk_norm_rope_bwd(dev["x"], dev["dy"], dx, dev["wq"], dev["wk"], dwq, dwk, dev["pos"], ws, q_heads=3,
                                 sections=(48,), **kw)

    def same():
        torch.cuda.synchronize()
        return all(torch.equal(a.cpu(), want[k]) for a, k in ((y, "y"), (dx, "dx"), (dwq, "dwq"), (dwk, "dwk")))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    step(stream=s)
    assert same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in (y, dx, dwq, dwk):
        t.fill_(float("nan"))
    graph.replay()
    assert same()
