"""The packed attention's waits running out, in the kernels that one CTA and that a cluster finishes. Under a wait budget
of zero a CTA's (or, of a cluster, its last one's) first tiles are not asked for: the call ends, sets MP_DEV_TIMEOUT,
stores no result that lacks a part, and leaves the context usable."""
import pytest
import torch

from gpu_util import mp, status_tensor
from test_gpu_attn_varlen import _cu, _inputs, _nan, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q_lens,k_lens,heads,kv", [
    ([300], [300], 2, 2),       # a CTA alone in all three kernels
    ([40], [4500], 2, 1),       # clusters share the keys (forward, dQ)
    ([1000], [1000], 8, 1),     # clusters share the queries (dK, dV)
])
@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("report", [True, False])
def test_waits_run_out(q_lens, k_lens, heads, kv, d, report, monkeypatch):
    cu_q, cu_k = _cu(q_lens), _cu(k_lens)
    Tq, Tk = sum(q_lens), sum(k_lens)
    inp = _inputs(Tq, Tk, heads, kv, d, seed=25000 + Tk)
    want = _run(inp, cu_q, cu_k, False)
    dev = {k: v.cuda() for k, v in inp.items()}
    cq, ck = cu_q.cuda(), cu_k.cuda()
    st = status_tensor()
    kw = dict(max_q=Tq, max_k=Tk, causal=False, d_status=st if report else None)
    O, lse, delta = _nan(Tq, heads, d), _nan(heads, Tq, dtype=torch.float32), _nan(heads, Tq, dtype=torch.float32)
    grads = [_nan(Tq, heads, d), _nan(Tk, kv, d), _nan(Tk, kv, d)]
    good_O, good_lse = want["O"].cuda(), want["LSE"].cuda()
    monkeypatch.setenv("MPTP_WAIT_BUDGET_NS", "0")
    mp().mp_attn_varlen_fwd(dev["Q"], dev["K"], dev["V"], O, lse, cq, ck, **kw)
    torch.cuda.synchronize()
    assert int(st.item()) == (mp().MP_DEV_TIMEOUT if report else 0)
    assert torch.isnan(O.float()).all() and torch.isnan(lse).all()
    st.zero_()
    mp().mp_attn_varlen_bwd(dev["Q"], dev["K"], dev["V"], good_O, good_lse, dev["dO"], *grads, delta, cq, ck, **kw)
    torch.cuda.synchronize()
    assert int(st.item()) == (mp().MP_DEV_TIMEOUT if report else 0)
    assert all(torch.isnan(g.float()).all() for g in grads)
    monkeypatch.delenv("MPTP_WAIT_BUDGET_NS")
    got = _run(inp, cu_q, cu_k, False)
    for k in want:
        assert torch.equal(got[k], want[k]), k
