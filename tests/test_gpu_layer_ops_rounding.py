"""The packed attention's and the gated block's errors are those of their roundings to bf16, no more.

One rounding's error, as a share of the norm, is measured on normally distributed values (0.0017); independent
roundings add in squares. Counted on each result's path:
  O, dV: P, the result; dQ, dK: O (through delta), dS, the result;
  Y, GU: the result; Z, dWd: Y, the result; dGU: U, G (whose weight in act' and act is about one), the result; dX, dW:
  those three and the result.
A quarter more is allowed for values that are not normal; twice the error fails."""
import math

import numpy as np
import pytest
import torch

import oracle
from gpu_util import f64, rel_fro
from test_gpu_attn_varlen import _cu, _inputs as attn_inputs, _run as attn_run
from test_gpu_glu import _inputs as glu_inputs, _run as glu_run

pytestmark = pytest.mark.gpu
_Z = torch.from_numpy(np.random.default_rng(26000).normal(size=1 << 18))
ONE = rel_fro(_Z.to(torch.bfloat16).double().numpy(), _Z.numpy())


def _bound(roundings):
    return 1.25 * math.sqrt(roundings) * ONE


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("q_lens,causal", [([777, 400], True), ([777, 400], False), ([1600], True)])
def test_attention_errors(q_lens, causal, d):
    cu = _cu(q_lens)
    inp = attn_inputs(sum(q_lens), sum(q_lens), 4, 2, d, seed=26100 + d)
    got = attn_run(inp, cu, cu, causal)
    x = {k: f64(v) for k, v in inp.items()}
    want = {"O": oracle.attn_varlen_fwd(x["Q"], x["K"], x["V"], cu.numpy(), cu.numpy(), causal, d ** -0.5)[0]}
    want.update(oracle.attn_varlen_bwd(x["Q"], x["K"], x["V"], x["dO"], cu.numpy(), cu.numpy(), causal, d ** -0.5))
    errs = {k: rel_fro(f64(got[k]), w) / _bound(2 if k in ("O", "dV") else 3) for k, w in want.items()}
    assert all(e <= 1.0 for e in errs.values()), errs


@pytest.mark.parametrize("T,h,f", [(9, 512, 1024), (300, 256, 1024), (1100, 128, 2176)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_block_errors(T, h, f, act):
    inp = glu_inputs(T, h, f, seed=26200)
    got = glu_run(inp, 2, act)
    x = {k: f64(v) for k, v in inp.items()}
    want = dict(zip(("GU", "Y", "Z"), oracle.glu_fwd(x["X"], x["W"], x["Wd"], act)))
    want.update(oracle.glu_bwd(x["X"], x["W"], x["Wd"], x["dZ"], act))
    count = {"GU": 1, "Y": 1, "Z": 2, "dWd": 2, "dGU": 3, "dX": 4, "dW": 4}
    errs = {k: rel_fro(f64(got[k].cpu()), want[k]) / _bound(count[k]) for k in want}
    assert all(e <= 1.0 for e in errs.values()), errs
