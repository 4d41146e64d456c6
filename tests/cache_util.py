"""Pools, page tables and inputs of the 8-bit cache for its tests."""
import numpy as np
import torch

F8 = torch.float8_e4m3fn


def ints(values):
    return torch.tensor(list(values), dtype=torch.int32)


def cu_of(lens):
    return ints(np.concatenate([[0], np.cumsum(lens)]))


def page_table(lens, page, seed, spare=2, room=0):
    """Pages of every sequence in a random order, `room` unused columns (-1) behind the longest; and the pool's size."""
    counts = [-(-int(n) // page) for n in lens]
    g = torch.Generator().manual_seed(seed)
    pages = max(1, sum(counts) + spare)
    order = torch.randperm(pages, generator=g).tolist()
    table = torch.full((len(counts), max(1, max(counts, default=0) + room)), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(counts):
        table[i, :n] = ints(order[at:at + n])
        at += n
    return table, pages


def pool(pages, kv, page, d, seed, spread=2, nan=False):
    """Codes [pages, 2, kv, page, d] (keys and values side by side) and scales [pages, 2, kv], powers of two that
    differ by 2^-spread .. 2^spread."""
    g = torch.Generator().manual_seed(seed)
    codes = (torch.randn(pages, 2, kv, page, d, generator=g) * 70).clamp(-448, 448).to(F8)
    if nan:  # pages and slots of nobody may hold anything
        codes.view(torch.uint8).fill_(0x7f)
    scales = torch.exp2(torch.randint(-spread, spread + 1, (pages, 2, kv), generator=g).float() - 6)
    return codes, scales


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()
