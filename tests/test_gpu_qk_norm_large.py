"""The norm of heads whose squares pass fp32's range, beside ordinary ones, against the float64 oracle: tolerances of
test_gpu_qk_norm, and half of bf16's least step (2^-134) where results come near it."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import f64
from test_gpu_qk_norm import EPS, _inputs, _pairs, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,nq,d", [(4, 3, 64), (20, 16, 128), (5, 4, 72), (2, 1, 256), (9, 9, 24)])
@pytest.mark.parametrize("e", [59, 63, 66, 90, 120])
def test_heads_beyond_the_range_of_their_squares(heads, nq, d, e):
    T, sec = 37, (d // 2 - d // 2 % 4,)
    inp = _inputs(T, heads, d, 1, 5000, 25100 + d)
    big = torch.rand(T, heads, 1, generator=torch.Generator().manual_seed(e)) < 0.4
    inp["x"] = torch.where(big, (inp["x"].float().clamp(-60, 60) * 2.0 ** e).to(torch.bfloat16), inp["x"])
    assert torch.isfinite(inp["x"]).all()
    got = _run(inp, nq, sections=sec)
    x, dy, wq, wk, pos = f64(inp["x"]), f64(inp["dy"]), f64(inp["wq"]), f64(inp["wk"]), inp["pos"].numpy()
    how = (pos, nq, sec, 10000.0, EPS)
    r = 1.0 / np.sqrt(np.mean(x * x, -1, keepdims=True) + EPS)
    n, w = x * r, np.stack([wq if h < nq else wk for h in range(heads)])
    y = oracle.qk_norm_rope(x, wq, wk, *how)
    assert np.all(np.abs(f64(got["y"]) - y) <= 2.0 ** -8 * np.abs(y) + 1e-5 * _pairs(n * w, sec, False))
    want = oracle.qk_norm_rope_bwd(x, dy, wq, wk, *how)
    g = _pairs(dy.copy(), sec, False)
    size = r * (np.abs(w) * g + np.abs(n) * np.mean(np.abs(w * n) * g, -1, keepdims=True))
    assert np.all(np.abs(f64(got["dx"]) - want["dx"]) <= 2.0 ** -8 * np.abs(want["dx"]) + 2e-5 * size + 2.0 ** -134)
    terms = (g * np.abs(n)).sum(0)
    for name, part in (("dwq", terms[:nq].sum(0)), ("dwk", terms[nq:].sum(0))):
        if np.any(part):
            assert np.all(np.abs(f64(got[name]) - want[name]) <= 2e-5 * part), name


def test_infinity_and_nan_stay_in_their_heads():
    inp = _inputs(9, 4, 64, 1, 50, 25200)
    clean = _run(inp, 3, sections=(32,))
    inp["x"][2, 1, 5], inp["x"][7, 3, 60] = float("inf"), float("nan")
    got = _run(inp, 3, sections=(32,))
    hit = torch.zeros(9, 4, dtype=torch.bool)
    hit[2, 1] = hit[7, 3] = True
    for k in ("y", "dx"):
        assert torch.isnan(got[k][hit]).any(-1).all() and torch.equal(got[k][~hit], clean[k][~hit])
    y = got["y"][2, 1]  # finite over infinite is zero, infinite over infinite NaN, in the element's pair alone
    assert torch.isnan(y[[5, 37]]).all() and not y[[i for i in range(64) if i not in (5, 37)]].any()
