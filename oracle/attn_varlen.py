"""Attention over packed sequences, forward and backward, float64. Test infrastructure.

Sequence n owns query rows [cu_q[n], cu_q[n+1]) and key rows [cu_k[n], cu_k[n+1]); query head j
reads key head j // (heads / kv_heads). Causal: the last query sees the last key, i.e. query i sees
keys 0 .. i + (nk - nq). O = softmax(scale Q K^T) V; a row that sees no key gives O = 0, log-sum-exp
-inf and no gradient. Rows outside every sequence stay 0.
"""
import numpy as np


def _sequences(cu_q, cu_k):
    for n in range(len(cu_q) - 1):
        yield slice(int(cu_q[n]), int(cu_q[n + 1])), slice(int(cu_k[n]), int(cu_k[n + 1]))


def _probabilities(q, k, causal, scale):
    """P [nq, nk] and the rows' log-sum-exp."""
    nq, nk = q.shape[0], k.shape[0]
    S = scale * (q @ k.T)
    if causal:
        S = np.where(np.arange(nk)[None, :] <= np.arange(nq)[:, None] + (nk - nq), S, -np.inf)
    if nk == 0:
        return np.zeros((nq, 0)), np.full(nq, -np.inf)
    m = S.max(axis=1, keepdims=True)
    m = np.where(np.isfinite(m), m, 0.0)
    e = np.exp(S - m)
    l = e.sum(axis=1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = (m + np.log(l))[:, 0]
    return e / np.where(l > 0, l, 1.0), lse


def attn_varlen_fwd(Q, K, V, cu_q, cu_k, causal, scale):
    """Q [Tq, heads, d], K, V [Tk, kv_heads, d] -> O [Tq, heads, d], LSE [heads, Tq]."""
    heads, group = Q.shape[1], Q.shape[1] // K.shape[1]
    O, LSE = np.zeros(Q.shape), np.full((heads, Q.shape[0]), -np.inf)
    for rq, rk in _sequences(cu_q, cu_k):
        for j in range(heads):
            P, lse = _probabilities(Q[rq, j], K[rk, j // group], causal, scale)
            O[rq, j], LSE[j, rq] = P @ V[rk, j // group], lse
    return O, LSE


def attn_varlen_bwd(Q, K, V, dO, cu_q, cu_k, causal, scale):
    """dict of dQ, dK, dV."""
    heads, group = Q.shape[1], Q.shape[1] // K.shape[1]
    g = {"dQ": np.zeros(Q.shape), "dK": np.zeros(K.shape), "dV": np.zeros(V.shape)}
    for rq, rk in _sequences(cu_q, cu_k):
        for j in range(heads):
            i = j // group
            P, _ = _probabilities(Q[rq, j], K[rk, i], causal, scale)
            dP = dO[rq, j] @ V[rk, i].T
            dS = P * (dP - (P * dP).sum(axis=1, keepdims=True))
            g["dQ"][rq, j] = scale * dS @ K[rk, i]
            g["dK"][rk, i] += scale * dS.T @ Q[rq, j]
            g["dV"][rk, i] += P.T @ dO[rq, j]
    return g
