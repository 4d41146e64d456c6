"""GPU parity of the rotation with several axes against the float64 oracle.

Tolerance per element: half a bf16 step of the result (2^-8 relative), plus the fp32 arithmetic and the
angle (within 2^-20 turns, 6e-6 radians) on the pair's two elements: 1e-5 (|a| + |b|)."""
import numpy as np
import pytest
import torch

import oracle
import synth
from gpu_util import f64, mp

pytestmark = pytest.mark.gpu


def _check(got, x, pos, sections, base, **kw):
    xr = f64(x)
    want = oracle.rope(xr, pos.numpy(), sections, base, **kw)
    n = sum(sections)
    size = np.zeros_like(xr)
    if kw.get("interleaved"):
        both = np.abs(xr[..., 0:2 * n:2]) + np.abs(xr[..., 1:2 * n:2])
        size[..., 0:2 * n:2] = size[..., 1:2 * n:2] = both
    else:
        size[..., :n] = size[..., n:2 * n] = np.abs(xr[..., :n]) + np.abs(xr[..., n:2 * n])
    err = np.abs(f64(got) - want)
    assert np.all(err <= 2.0 ** -8 * np.abs(want) + 1e-5 * size), float(err.max())


def _pos(axes, T, top, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, top, (axes, T), generator=g, dtype=torch.int64).to(torch.int32)


@pytest.mark.parametrize("T,heads,d,sections,base,top", [
    (1, 1, 8, (4,), 10000.0, 100),               # one token, one head, one group of pairs
    (5, 3, 64, (16, 8, 8), 10000.0, 1 << 20),
    (257, 40, 128, (16, 24, 24), 1e6, 40000),
    (33, 7, 96, (16, 16, 16), 10000.0, 2147483647),  # the farthest positions
    (100, 5, 72, (0, 18, 18), 100.0, 300),       # an axis without pairs; 8-byte pieces
    (64, 3, 80, (20, 9, 3), 10000.0, 5000),      # 16 elements of each head pass through
    (19, 2, 256, (32, 32, 32, 32), 500.0, 999),  # four axes, the widest head
    (9, 70, 16, (1, 2, 1), 0.5, 64),             # base below 1: faster than a radian a step
    (3000, 2, 64, (32,), 10000.0, 3000),
])
@pytest.mark.parametrize("interleaved,per_axis,inverse", [(False, False, False), (True, True, True),
                                                          (False, True, False), (True, False, False)])
def test_rope_matches_oracle(T, heads, d, sections, base, top, interleaved, per_axis, inverse):
    x = synth.normal_bf16((T, heads, d), 1.0, 20000 + T + d)
    pos = _pos(len(sections), T, top, 20001 + T)
    y = torch.full((T, heads, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    kw = dict(interleaved=interleaved, per_axis=per_axis, inverse=inverse)
    mp().mp_rope_axes(x.cuda(), y, pos.cuda(), sections=sections, base=base, **kw)
    _check(y.cpu(), x, pos, sections, base, **kw)


def test_rope_negative_positions():
    x = synth.normal_bf16((50, 4, 64), 1.0, 20100)
    pos = _pos(2, 50, 1 << 20, 20101) - (1 << 19)
    pos[0, 0] = -2147483648
    y = torch.empty_like(x, device="cuda")
    mp().mp_rope_axes(x.cuda(), y, pos.cuda(), sections=(20, 12))
    _check(y.cpu(), x, pos, (20, 12), 10000.0)


def test_rope_strided_rows_and_in_place():
    # queries and keys inside packed projection rows; nothing else in the rows changes
    qkv = synth.normal_bf16((77, 9, 64), 1.0, 20200)
    pos = _pos(3, 77, 1000, 20201)
    dev = qkv.cuda()
    out = torch.full((77, 12, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    mp().mp_rope_axes(dev[:, 1:7], out[:, 2:8], pos.cuda(), sections=(8, 12, 12))
    _check(out[:, 2:8].cpu(), qkv[:, 1:7], pos, (8, 12, 12), 10000.0)
    assert torch.all(out[:, :2] == 3.0) and torch.all(out[:, 8:] == 3.0)
    mp().mp_rope_axes(dev[:, 1:7], dev[:, 1:7], pos.cuda(), sections=(8, 12, 12))
    assert torch.equal(dev[:, 1:7], out[:, 2:8])
    assert torch.equal(dev[:, 0].cpu(), qkv[:, 0]) and torch.equal(dev[:, 7:].cpu(), qkv[:, 7:])


def test_rope_back_and_forth_returns_the_input():
    # two roundings of at most half a step of the pair's length (2^-8 of |a| + |b|, twice)
    x = synth.normal_bf16((64, 4, 96), 1.0, 20300)
    pos = _pos(3, 64, 100000, 20301).cuda()
    y, z = torch.empty_like(x, device="cuda"), torch.empty_like(x, device="cuda")
    mp().mp_rope_axes(x.cuda(), y, pos, sections=(16, 16, 16))
    mp().mp_rope_axes(y, z, pos, sections=(16, 16, 16), inverse=True)
    pair = (x[..., :48].abs() + x[..., 48:].abs()).double().repeat(1, 1, 2)
    assert torch.all((z.cpu().double() - x.double()).abs() <= 2 * 2.0 ** -8 * pair + 1e-5)


def test_rope_empty_batch_and_other_stream():
    x = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    mp().mp_rope_axes(x, x, torch.empty(1, 0, dtype=torch.int32, device="cuda"), sections=(32,))
    xs = synth.normal_bf16((31, 2, 64), 1.0, 20400)
    pos = _pos(1, 31, 50, 20401)
    s = torch.cuda.Stream()
    dev, p = xs.cuda(), pos.cuda()
    y = torch.empty_like(dev)
    s.wait_stream(torch.cuda.current_stream())
    mp().mp_rope_axes(dev, y, p, sections=(32,), stream=s)
    s.synchronize()
    _check(y.cpu(), xs, pos, (32,), 10000.0)


@pytest.mark.parametrize("base", [2.0, 1.0, 0.5, 0.01])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope_farthest_positions_at_small_bases(base, inverse):
    # Angles from 80 decimal digits: within 2^-20 turns, or 2^-20 / base where the base is below 1; on the pair's two
    # elements as radians, with half a bf16 step of the result and the fp32 arithmetic (three roundings, 2^-24 each).
    from decimal import Decimal, getcontext
    getcontext().prec = 80
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534")
    n, pos = 48, [2147483647, -2147483648, 2147480001, 1999999973, -1234567891, 77]
    turns = np.zeros((len(pos), n))
    for i in range(n):
        f = Decimal(base) ** (-Decimal(i) / Decimal(n)) / two_pi
        for k, p in enumerate(pos):
            t = p * f
            turns[k, i] = float(t - t.to_integral_value())
    ang = 2 * np.pi * turns * (-1 if inverse else 1)
    x = synth.normal_bf16((len(pos), 3, 2 * n), 1.0, 20500)
    y = torch.empty(len(pos), 3, 2 * n, dtype=torch.bfloat16, device="cuda")
    mp().mp_rope_axes(x.cuda(), y, torch.tensor([pos], dtype=torch.int32, device="cuda"), sections=(n,), base=base,
                      inverse=inverse)
    a, b = f64(x)[..., :n], f64(x)[..., n:]
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    want = np.concatenate([a * c - b * s, b * c + a * s], -1)
    size = np.concatenate([np.abs(a) + np.abs(b)] * 2, -1)
    tol = 2.0 ** -8 * np.abs(want) + (2 * np.pi * 2.0 ** -20 / min(base, 1.0) + 2.0 ** -22) * size
    assert np.all(np.abs(f64(y.cpu()) - want) <= tol)
