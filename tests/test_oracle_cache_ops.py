"""Pins of the oracle of the query and key norm, the 8-bit cache and the attention over it (CPU only)."""
import numpy as np
import torch

import oracle


def test_e4m3_rounding_matches_torch_and_ties_go_to_even():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    finite = codes[np.isfinite(codes)]
    assert np.array_equal(oracle.e4m3_round(finite), finite)
    g = torch.Generator().manual_seed(1)
    x = torch.randn(20000, generator=g) * torch.exp(3 * torch.randn(20000, generator=g))
    x = x.clamp(-448, 448)
    assert np.array_equal(oracle.e4m3_round(x.numpy()), x.to(torch.float8_e4m3fn).double().numpy())
    # 17 lies between 16 and 18 (codes 0x58, 0x59), 2^-10 between 0 and the smallest subnormal
    assert oracle.e4m3_round(17.0) == 16.0 and oracle.e4m3_round(19.0) == 20.0
    assert oracle.e4m3_round(2.0 ** -10) == 0.0 and oracle.e4m3_round(3 * 2.0 ** -10) == 2.0 ** -8
    assert oracle.e4m3_round(1e9) == 448.0 and np.isnan(oracle.e4m3_round(np.inf))


def test_page_scale_is_the_smallest_power_of_two():
    assert oracle.page_scale(np.array([448.0])) == 1.0
    assert oracle.page_scale(np.array([448.5, -1.0])) == 2.0
    assert oracle.page_scale(np.array([0.0])) == 2.0 ** -100
    assert oracle.page_scale(np.array([np.inf, np.nan, 3.5])) == 2.0 ** -7


def test_norm_gradients_match_differences():
    rng = np.random.default_rng(2)
    T, heads, nq, d, sections = 3, 3, 2, 16, (2, 4)
    x, dy = rng.normal(size=(T, heads, d)), rng.normal(size=(T, heads, d))
    wq, wk, pos = rng.normal(size=d), rng.normal(size=d), rng.integers(0, 50, size=(2, T))
    for kw in (dict(), dict(interleaved=True, per_axis=True)):
        def loss(x, wq, wk):
            return float((oracle.qk_norm_rope(x, wq, wk, pos, nq, sections, 100.0, 1e-3, **kw) * dy).sum())
        got = oracle.qk_norm_rope_bwd(x, dy, wq, wk, pos, nq, sections, 100.0, 1e-3, **kw)
        for name, i in (("dx", 0), ("dwq", 1), ("dwk", 2)):
            args = [x, wq, wk]
            for at in list(np.ndindex(args[i].shape))[::5]:
                e = np.zeros_like(args[i])
                e[at] = 1e-5
                up, down = ([*args[:i], args[i] + s * e, *args[i + 1:]] for s in (1, -1))
                assert abs((loss(*up) - loss(*down)) / 2e-5 - got[name][at]) < 1e-7


def test_norm_of_a_unit_head_is_the_rotation_and_of_zeros_is_zero():
    x = np.ones((1, 1, 8)) * np.array([1, -1, 1, -1, 1, -1, 1, -1.0])
    y = oracle.qk_norm_rope(x, np.ones(8), None, np.array([[5]]), 1, (4,), 10.0, 1e-12)
    assert np.allclose(y, oracle.rope(x, np.array([[5]]), (4,), 10.0), atol=1e-11)
    assert not oracle.qk_norm_rope(0 * x, np.ones(8), None, np.array([[5]]), 1, (4,), 10.0, 1e-12).any()


def test_cache_filled_token_by_token_equals_one_filled_at_once_where_no_scale_grows():
    rng = np.random.default_rng(3)
    x = rng.normal(size=(37, 2, 16)).clip(-1.9, 1.9)
    x[0] = 1.95  # the page's largest values come first
    x[16], x[32] = -1.95, 1.95
    table, codes, scales = [[2, 0, 3]], [np.zeros((4, 2, 16, 16)) for _ in range(2)], [np.zeros((4, 2)) for _ in range(2)]
    oracle.kv_cache_write(x, codes[0], scales[0], table, [0, 37], [0], 16)
    for k in range(37):
        oracle.kv_cache_write(x[k:k + 1], codes[1], scales[1], table, [0, 1], [k], 16)
    assert np.array_equal(codes[0], codes[1]) and np.array_equal(scales[0], scales[1])
    back = oracle.kv_cache_rows(codes[0], scales[0], table[0], 16, 0, 37)
    assert np.all(np.abs(back - x) <= 2.0 ** -4 * np.abs(x) + 2.0 ** -10 * scales[0].max())


def test_a_growing_scale_keeps_old_values_but_those_that_become_subnormal():
    codes, scales = np.zeros((1, 1, 16, 16)), np.zeros((1, 1))
    old = np.linspace(0.01, 1.0, 16).reshape(1, 1, 16)
    oracle.kv_cache_write(old, codes, scales, [[0]], [0, 1], [0], 16)
    was = codes[0, 0, 0] * scales[0, 0]
    oracle.kv_cache_write(8.0 * np.ones((1, 1, 16)), codes, scales, [[0]], [0, 1], [1], 16)
    assert scales[0, 0] == 2.0 ** -5 and np.array_equal(codes[0, 0, 0] * scales[0, 0], was)


def test_attention_over_the_cache_is_the_attention_of_its_values():
    rng = np.random.default_rng(4)
    kc, vc = (oracle.e4m3_round(rng.normal(size=(3, 1, 16, 16)) * 60) for _ in range(2))
    s = np.full((3, 1), 2.0 ** -6)
    Q = rng.normal(size=(2, 2, 16))
    O, LSE = oracle.attn_cache_fwd(Q, kc, vc, s, s, [[2, 0], [1, 1]], [0, 1, 2], [20, 0], 16, True, 0.25)
    k = np.concatenate([kc[2, 0], kc[0, 0]])[:20] / 64
    v = np.concatenate([vc[2, 0], vc[0, 0]])[:20] / 64
    p = np.exp(0.25 * Q[0, 1] @ k.T)
    assert np.allclose(O[0, 1], p @ v / p.sum()) and np.isclose(LSE[1, 0], np.log(p.sum()))
    assert not O[1].any() and np.all(LSE[:, 1] == -np.inf)
