"""Gated feed-forward block, forward and backward, float64. Test infrastructure.

G = X Wg, U = X Wu, Y = act(G) * U, Z = Y Wd with W = [Wg | Wu]; act is SiLU g / (1 + e^-g) or the
erf GeLU. Backward: dY = dZ Wd^T, dG = dY U act'(G), dU = dY act(G), dX = [dG | dU] W^T,
dW = X^T [dG | dU], dWd = Y^T dZ. ``glu_sharded_fwd`` cuts gate and up by the same columns per shard
and sums the shards' partial outputs.
"""
import numpy as np

from .gelu import gelu, gelu_prime


def glu_act(g, act):
    """(act(g), act'(g))."""
    g = np.asarray(g, dtype=np.float64)
    if act == "gelu":
        return gelu(g), gelu_prime(g)
    s = np.where(g >= 0, 1.0 / (1.0 + np.exp(-np.abs(g))), np.exp(-np.abs(g)) / (1.0 + np.exp(-np.abs(g))))
    return g * s, s * (1.0 + g * (1.0 - s))


def glu_fwd(X, W, Wd, act):
    """(GU, Y, Z)."""
    f = Wd.shape[0]
    GU = X @ W
    Y = glu_act(GU[:, :f], act)[0] * GU[:, f:]
    return GU, Y, Y @ Wd


def glu_bwd(X, W, Wd, dZ, act):
    """dict of dX, dW, dWd, dGU."""
    f = Wd.shape[0]
    GU, Y, _ = glu_fwd(X, W, Wd, act)
    a, da = glu_act(GU[:, :f], act)
    dY = dZ @ Wd.T
    dGU = np.concatenate([dY * GU[:, f:] * da, dY * a], axis=1)
    return {"dX": dGU @ W.T, "dW": X.T @ dGU, "dWd": Y.T @ dZ, "dGU": dGU}


def glu_sharded_fwd(X, W, Wd, act, t):
    """Z as the sum of t shards' partial outputs."""
    f = Wd.shape[0]
    fs = f // t
    Z = np.zeros((X.shape[0], Wd.shape[1]))
    for i in range(t):
        c = slice(i * fs, (i + 1) * fs)
        G, U = X @ W[:, :f][:, c], X @ W[:, f:][:, c]
        Z += (glu_act(G, act)[0] * U) @ Wd[c]
    return Z
