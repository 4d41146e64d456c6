"""A transformer layer's training step on packed video clips and texts, with the library's kernels.

    python examples/gated_layer_step.py [--steps 5]

    q, k, v = X Wqkv                       (torch; key heads shared by groups of query heads)
    q, k    = rotated by time, row, column (mp_rope_axes)
    a       = attention within sequences   (mp_attn_varlen_fwd / _bwd)
    H       = X + a Wo                     (torch)
    Y       = H + (act(H Wg) * (H Wu)) Wd  (mp_glu_fwd / _bwd)
    loss    = mean((Y - target)^2) / 2

A step goes down h times its gradient, that of the tokens' mean squared error.
The layer has no normalisation, to keep to the point. Every buffer is made once, in `Layer`; a step
allocates only torch's matrix products.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import tensor_transformer_layer_gb300 as mp  # noqa: E402

BF16 = torch.bfloat16


def clip_positions(frames, rows, cols):
    """[3, frames * rows * cols] positions of a clip's patches, time first."""
    t, y, x = torch.meshgrid(torch.arange(frames), torch.arange(rows), torch.arange(cols), indexing="ij")
    return torch.stack([t.flatten(), y.flatten(), x.flatten()])


def text_positions(n):
    """A text's tokens stand on the diagonal: the three axes advance together."""
    return torch.arange(n).expand(3, n)


class Layer:
    def __init__(self, positions, heads=8, kv_heads=2, d=64, f=1024, sections=(8, 12, 12), t=2, causal=False, seed=0):
        self.heads, self.kv, self.d, self.f, self.t, self.causal, self.sections = heads, kv_heads, d, f, t, causal, sections
        self.h = heads * d
        lens = [p.shape[1] for p in positions]
        self.T, self.longest = sum(lens), max(lens)
        cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
        self.cu, self.pos = cu.cuda(), torch.cat(positions, 1).to(torch.int32).contiguous().cuda()
        g = torch.Generator(device="cuda").manual_seed(seed)

        def w(*shape):
            return (torch.randn(*shape, generator=g, device="cuda") * shape[0] ** -0.5).to(BF16)

        n = heads + 2 * kv_heads
        self.Wqkv, self.Wo, self.W, self.Wd = w(self.h, n * d), w(self.h, self.h), w(self.h, 2 * f), w(f, self.h)

        def e(*shape, dtype=BF16):
            return torch.empty(*shape, device="cuda", dtype=dtype)

        T, h = self.T, self.h
        self.qkv, self.dqkv = e(T, n, d), e(T, n, d)
        self.O, self.dO = e(T, heads, d), e(T, heads, d)
        self.lse, self.delta = e(heads, T, dtype=torch.float32), e(heads, T, dtype=torch.float32)
        self.Z, self.Y, self.GU, self.dGU = e(T, h), e(T, f), e(T, 2 * f), e(T, 2 * f)
        self.dH, self.dW, self.dWd = e(T, h), e(h, 2 * f), e(f, h)
        self.status = torch.zeros(1, device="cuda", dtype=torch.int32)

    def _parts(self, x):
        return x[:, :self.heads], x[:, self.heads:self.heads + self.kv], x[:, self.heads + self.kv:]

    def forward(self, X):
        torch.matmul(X, self.Wqkv, out=self.qkv.view(self.T, -1))
        qk = self.qkv[:, :self.heads + self.kv]
        mp.mp_rope_axes(qk, qk, self.pos, sections=self.sections)  # in place, in the packed rows
        q, k, v = self._parts(self.qkv)
        mp.mp_attn_varlen_fwd(q, k, v, self.O, self.lse, self.cu, self.cu, max_q=self.longest, max_k=self.longest,
                              causal=self.causal, d_status=self.status)
        self.H = X + self.O.view(self.T, self.h) @ self.Wo
        mp.mp_glu_fwd(self.H, self.W, self.Wd, self.Z, self.Y, self.GU, t=self.t, d_status=self.status)
        return self.H + self.Z

    def backward(self, X, dY):
        """Gradients of the weights and of X for the last forward."""
        mp.mp_glu_bwd(self.H, self.W, self.Wd, self.GU, self.Y, dY, self.dH, self.dW, self.dWd, self.dGU, t=self.t,
                      d_status=self.status)
        dH = self.dH + dY
        o = self.O.view(self.T, self.h)
        dWo = o.t() @ dH
        torch.matmul(dH, self.Wo.t(), out=self.dO.view(self.T, self.h))
        q, k, v = self._parts(self.qkv)
        dq, dk, dv = self._parts(self.dqkv)
        mp.mp_attn_varlen_bwd(q, k, v, self.O, self.lse, self.dO, dq, dk, dv, self.delta, self.cu, self.cu,
                              max_q=self.longest, max_k=self.longest, causal=self.causal, d_status=self.status)
        dqk = self.dqkv[:, :self.heads + self.kv]
        mp.mp_rope_axes(dqk, dqk, self.pos, sections=self.sections, inverse=True)
        flat = self.dqkv.view(self.T, -1)
        return {"Wqkv": X.t() @ flat, "Wo": dWo, "W": self.dW, "Wd": self.dWd, "X": dH + flat @ self.Wqkv.t()}

    def step(self, X, target, lr):
        """One step of gradient descent; the loss before it."""
        err = self.forward(X) - target
        grads = self.backward(X, err / err.numel() * self.h)
        for name in ("Wqkv", "Wo", "W", "Wd"):
            getattr(self, name).sub_(lr * grads[name])
        return 0.5 * err.float().square().mean()


def main(steps=5):
    layer = Layer([clip_positions(4, 9, 16), text_positions(77), clip_positions(1, 12, 21), text_positions(1)])
    g = torch.Generator(device="cuda").manual_seed(1)
    X, target = (torch.randn(layer.T, layer.h, generator=g, device="cuda").to(BF16) for _ in range(2))
    losses = [float(layer.step(X, target, lr=0.1)) for _ in range(steps)]
    code = mp.mp_status_from_device(int(layer.status.item()))
    if code != mp.MP_OK:
        raise mp.MptpError("gated_layer_step", code)
    print("tokens", layer.T, "losses", " ".join(f"{x:.4f}" for x in losses))
    return losses


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    p.add_argument("--steps", type=int, default=5)
    main(p.parse_args().steps)
