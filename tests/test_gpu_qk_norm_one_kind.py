"""The norm's backward where all heads are queries, or all are keys: the other weight's gradient is a sum over no heads."""
import pytest
import torch

import synth
from gpu_util import mp

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,heads,d", [(1, 1, 8), (40, 4, 64), (1250, 40, 128), (3001, 2, 72), (0, 3, 64)])
@pytest.mark.parametrize("queries", [True, False])
def test_gradient_of_the_weight_that_no_head_takes_is_zero(T, heads, d, queries):
    nq = heads if queries else 0
    x, dy = (synth.normal_bf16((T, heads, d), 1.0, 25000 + k).cuda() for k in (0, 1))
    w = synth.normal_bf16((2, d), 1.0, 25002).cuda()
    pos = torch.arange(T, dtype=torch.int32, device="cuda")[None]
    ws = torch.full((max(4, mp().mp_qk_norm_rope_bwd_workspace_bytes(T, heads, d)),), 0xff, dtype=torch.uint8, device="cuda")

    def run(both):
        dx = torch.empty_like(x)
        dw = torch.full((2, d), float("nan"), device="cuda")
        mp().mp_qk_norm_rope_bwd(x, dy, dx, w[0] if both or queries else None, w[1] if both or not queries else None,
                                 dw[0] if both or queries else None, dw[1] if both or not queries else None, pos, ws.clone(),
                                 q_heads=nq, sections=(d // 2,))
        return dx, dw

    (dx, dw), (want_dx, want_dw) = run(True), run(False)
    used, other = (0, 1) if queries else (1, 0)
    assert not dw[other].any()
    assert torch.equal(dw[used], want_dw[used]) and torch.isfinite(dw).all() and torch.equal(dx, want_dx)
