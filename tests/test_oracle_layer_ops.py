"""Pins of the oracles of the rotation with several axes, the gated block and the packed attention:
finite differences of every gradient, closed forms, and the older oracles that they reduce to."""
import numpy as np
import pytest

import oracle


def _diff(f, x, eps=1e-6):
    """Central differences of a scalar function of an array."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += eps
        b[i] -= eps
        g[i] = (f(a) - f(b)) / (2 * eps)
    return g


def test_rope_one_axis_closed_form():
    # base^0 = 1: pair 0 of a head turns by its position in radians.
    x = np.zeros((3, 1, 8))
    x[:, 0, 0] = 1.0
    y = oracle.rope(x, np.array([[0, 1, 2]]), [4], 10000.0)
    assert np.allclose(y[:, 0, 0], np.cos([0, 1, 2])) and np.allclose(y[:, 0, 4], np.sin([0, 1, 2]))
    y = oracle.rope(x, np.array([[0, 1, 2]]), [4], 10000.0, interleaved=True)
    assert np.allclose(y[:, 0, 1], np.sin([0, 1, 2]))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("per_axis", [False, True])
def test_rope_gradient_is_the_inverse(interleaved, per_axis):
    rng = np.random.default_rng(1)
    x, w = rng.normal(size=(2, 2, 20)), rng.normal(size=(2, 2, 20))
    pos = np.array([[3, 100], [7, 0], [1, 9]])
    kw = dict(interleaved=interleaved, per_axis=per_axis)
    num = _diff(lambda z: float((oracle.rope(z, pos, [2, 1, 5], 100.0, **kw) * w).sum()), x)
    assert np.allclose(num, oracle.rope(w, pos, [2, 1, 5], 100.0, inverse=True, **kw), atol=1e-7)
    y = oracle.rope(x, pos, [2, 1, 5], 100.0, **kw)
    assert np.allclose(oracle.rope(y, pos, [2, 1, 5], 100.0, inverse=True, **kw), x)
    assert np.allclose(y[..., 16:], x[..., 16:])


def test_rope_scores_depend_on_differences_only():
    rng = np.random.default_rng(2)
    q, k = rng.normal(size=(1, 1, 16)), rng.normal(size=(1, 1, 16))

    def score(pq, pk):
        a = oracle.rope(q, np.array(pq)[:, None], [3, 5], 50.0)
        b = oracle.rope(k, np.array(pk)[:, None], [3, 5], 50.0)
        return float((a * b).sum())

    assert abs(score([5, 9], [2, 4]) - score([105, 1009], [102, 1004])) < 1e-9


def test_glu_act_values():
    a, da = oracle.glu_act(np.array([0.0, 800.0, -800.0]), "silu")
    assert np.allclose(a, [0.0, 800.0, 0.0]) and np.allclose(da, [0.5, 1.0, 0.0])
    assert np.isfinite(a).all()


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_glu_gradients_by_differences(act):
    rng = np.random.default_rng(3)
    X, W, Wd, dZ = (rng.normal(size=s) for s in ((3, 4), (4, 10), (5, 4), (3, 4)))
    g = oracle.glu_bwd(X, W, Wd, dZ, act)
    assert np.allclose(g["dX"], _diff(lambda z: float((oracle.glu_fwd(z, W, Wd, act)[2] * dZ).sum()), X), atol=1e-6)
    assert np.allclose(g["dW"], _diff(lambda z: float((oracle.glu_fwd(X, z, Wd, act)[2] * dZ).sum()), W), atol=1e-6)
    assert np.allclose(g["dWd"], _diff(lambda z: float((oracle.glu_fwd(X, W, z, act)[2] * dZ).sum()), Wd), atol=1e-6)


def test_glu_shards_sum_to_the_whole():
    rng = np.random.default_rng(4)
    X, W, Wd = (rng.normal(size=s) for s in ((3, 6), (6, 16), (8, 6)))
    want = oracle.glu_fwd(X, W, Wd, "silu")[2]
    for t in (1, 2, 4):
        assert np.allclose(oracle.glu_sharded_fwd(X, W, Wd, "silu", t), want)


def test_attn_varlen_reduces_to_the_block_oracle():
    rng = np.random.default_rng(5)
    b, s, heads, d = 2, 6, 3, 4
    qkv = rng.normal(size=(b * s, 3 * heads * d))
    w = heads * d
    want = oracle.attention_heads(qkv[:, :w], qkv[:, w:2 * w], qkv[:, 2 * w:], heads, b, s)
    Q, K, V = (qkv[:, i * heads * d:(i + 1) * heads * d].reshape(b * s, heads, d) for i in range(3))
    cu = [0, s, 2 * s]
    O, LSE = oracle.attn_varlen_fwd(Q, K, V, cu, cu, True, 1.0 / np.sqrt(d))
    assert np.allclose(O.reshape(b * s, -1), want)
    assert np.allclose(LSE[:, 0], (Q[0] * K[0]).sum(-1) / np.sqrt(d))  # a first row sees one key


@pytest.mark.parametrize("causal", [False, True])
def test_attn_varlen_gradients_by_differences(causal):
    # shared key heads, a sequence without keys, one without queries, rows that see nothing
    rng = np.random.default_rng(6)
    cu_q, cu_k = [0, 3, 5, 5, 9], [0, 4, 4, 6, 8]
    Q, dO = rng.normal(size=(10, 4, 3)), rng.normal(size=(10, 4, 3))
    K, V = rng.normal(size=(8, 2, 3)), rng.normal(size=(8, 2, 3))
    g = oracle.attn_varlen_bwd(Q, K, V, dO, cu_q, cu_k, causal, 0.7)

    def loss(q, k, v):
        return float((oracle.attn_varlen_fwd(q, k, v, cu_q, cu_k, causal, 0.7)[0] * dO).sum())

    assert np.allclose(g["dQ"], _diff(lambda z: loss(z, K, V), Q), atol=1e-7)
    assert np.allclose(g["dK"], _diff(lambda z: loss(Q, z, V), K), atol=1e-7)
    assert np.allclose(g["dV"], _diff(lambda z: loss(Q, K, z), V), atol=1e-7)


def test_attn_varlen_rows_without_keys():
    rng = np.random.default_rng(7)
    Q, K = rng.normal(size=(4, 1, 2)), rng.normal(size=(2, 1, 2))
    O, LSE = oracle.attn_varlen_fwd(Q, K, K, [0, 4], [0, 2], True, 1.0)
    assert np.all(O[:2] == 0) and np.all(np.isneginf(LSE[0, :2])) and np.isfinite(LSE[0, 2:]).all()
