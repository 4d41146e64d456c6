"""The kernels of a decoding step may start while the kernel before them is still writing, and wait for it inside. Loads that
promise memory which is read-only for a kernel's whole life (the non-coherent path) may see what was there before, so none
of these kernels makes that promise."""
import os
import re

import pytest
import torch

from tensor_transformer_layer_gb300 import build


@pytest.mark.parametrize("name", ["mptp_attn_cache.cu", "mptp_kv_cache.cu", "mptp_kv_cache.cuh", "mptp_qk_norm.cu", "mptp_rope.cuh"])
def test_no_load_promises_read_only_memory(name):
    with open(os.path.join(build.CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    assert not re.findall(r"__ldg|__restrict__|\bld\.global\.nc\b|\.nc\b", text)


@pytest.mark.gpu
def test_lengths_offsets_and_pages_written_by_the_kernel_before():
    """Offsets, lengths and the page table come from a kernel that lets the next one start early; two sets in turn."""
    import tensor_transformer_layer_gb300 as mp
    nseq, heads, kv, d, page = 3, 4, 2, 64, 16
    g = torch.Generator().manual_seed(7)
    codes = (torch.randn(40, 2, kv, page, d, generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn).cuda()
    scales = torch.full((40, 2, kv), 2.0 ** -6, device="cuda")
    Q = torch.randn(6, heads, d, generator=g).to(torch.bfloat16).cuda()
    # an embedding's rows of 64 values hold 32 integers: offsets, lengths, then a table's rows; rows 0 .. 4 one set, 5 .. 9 another
    sets = torch.zeros(10, 32, dtype=torch.int32)
    sets[0, :4], sets[5, :4] = torch.tensor([0, 1, 3, 6]), torch.tensor([0, 4, 4, 6])
    sets[1, :3], sets[6, :3] = torch.tensor([300, 7, 40]), torch.tensor([9, 512, 130])
    for first in (2, 7):
        for i in range(nseq):
            sets[first + i] = torch.randperm(40, generator=g)[:32].to(torch.int32)
    E = torch.zeros(128, 64, dtype=torch.bfloat16)
    E[:10] = sets.view(torch.bfloat16)
    E = E.cuda()
    ids = [torch.arange(5, dtype=torch.int32).cuda(), torch.arange(5, 10, dtype=torch.int32).cuda()]
    ws = torch.empty(mp.mp_attn_cache_workspace_bytes(heads, kv, d, 4), dtype=torch.uint8, device="cuda")

    def step(now, which, O, LSE):
        mp.mp_vocab_embed(ids[which], E, now, v_valid=128, t=1)
        ints = now.view(torch.int32)
        mp.mp_attn_cache_fwd(Q, codes[:, 0], codes[:, 1], scales[:, 0], scales[:, 1], O, LSE, ints[2:5], ints[0, :4], ints[1, :3],
                             ws, max_q=4)

    want, got = [], []
    for which in (0, 1):
        now, O, LSE = torch.empty(5, 64, dtype=torch.bfloat16, device="cuda"), torch.empty_like(Q), torch.empty(4, 6, device="cuda")
        step(now, which, O, LSE)
        torch.cuda.synchronize()
        want.append((O, LSE))
    now = torch.zeros(5, 64, dtype=torch.bfloat16, device="cuda")
    outs = [(torch.empty_like(Q), torch.empty(4, 6, device="cuda")) for _ in range(100)]
    torch.cuda.synchronize()
    for k, (O, LSE) in enumerate(outs):
        step(now, k % 2, O, LSE)
    torch.cuda.synchronize()
    for k, (O, LSE) in enumerate(outs):
        assert torch.equal(O, want[k % 2][0]) and torch.equal(LSE, want[k % 2][1]), k
    assert not torch.equal(want[0][0], want[1][0])
