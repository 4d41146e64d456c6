"""The example's layer step against the same layer in torch autograd (float64 from the same bf16 values).

Tolerance: every value on the longest path (qkv, rotated q and k, P or dS, O, H, gates, dGU, dH, dO, the
gradient itself) is rounded to bf16 once, some twice: sqrt(12) roundings of half a step, 2^-8 each."""
import math
import os
import sys

import pytest
import torch


pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
TOL = math.sqrt(12) * 2.0 ** -8


def _rotate(x, pos, sections, base=10000.0):
    n = sum(sections)
    axis = torch.repeat_interleave(torch.arange(len(sections), device=x.device), torch.tensor(sections, device=x.device))
    ang = pos.double()[axis].t() * base ** (-torch.arange(n, device=x.device, dtype=torch.float64) / n)
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    a, b = x[..., :n], x[..., n:2 * n]
    return torch.cat([a * c - b * s, b * c + a * s, x[..., 2 * n:]], -1)


def _plain(layer, X, W):
    T, h, kv, d = layer.T, layer.heads, layer.kv, layer.d
    qkv = (X @ W["Wqkv"]).view(T, h + 2 * kv, d)
    qk = _rotate(qkv[:, :h + kv], layer.pos, layer.sections)
    q, k, v = qk[:, :h], qk[:, h:].repeat_interleave(h // kv, 1), qkv[:, h + kv:].repeat_interleave(h // kv, 1)
    cu, out = layer.cu.tolist(), []
    for a, b in zip(cu, cu[1:]):
        s = torch.einsum("ihd,jhd->hij", q[a:b], k[a:b]) / math.sqrt(d)
        if layer.causal:
            s = s.masked_fill(torch.ones_like(s[0], dtype=torch.bool).triu(1), -math.inf)
        out.append(torch.einsum("hij,jhd->ihd", s.softmax(-1), v[a:b]))
    H = X + torch.cat(out).reshape(T, h * d) @ W["Wo"]
    g, u = (H @ W["W"]).chunk(2, 1)
    return H + (torch.nn.functional.silu(g) * u) @ W["Wd"]


@pytest.mark.parametrize("causal", [False, True])
def test_layer_step_matches_autograd(causal):
    import gated_layer_step as ex
    layer = ex.Layer([ex.clip_positions(3, 5, 7), ex.text_positions(33), ex.text_positions(1), ex.clip_positions(1, 12, 13)],
                     causal=causal, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    X, dY = (torch.randn(layer.T, layer.h, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    W = {k: getattr(layer, k).double().requires_grad_() for k in ("Wqkv", "Wo", "W", "Wd")}
    x = X.double().requires_grad_()
    want = _plain(layer, x, W)
    grads = torch.autograd.grad(want, [x] + list(W.values()), dY.double())
    ref = dict(zip(["X"] + list(W), grads))
    got = layer.forward(X)
    out = layer.backward(X, dY)
    assert int(layer.status.item()) == 0

    def far(a, b):
        return float((a.double() - b).norm() / b.norm())

    assert far(got, want.detach()) <= TOL
    errs = {k: far(out[k], ref[k]) for k in ref}
    assert all(v <= TOL for v in errs.values()), errs


def test_example_runs_and_learns():
    import gated_layer_step as ex
    losses = ex.main(steps=4)
    assert all(math.isfinite(x) for x in losses) and losses[-1] < losses[0]
