"""Measured cases of the operators around an 8-bit key and value cache: the norm of queries and keys with their
rotation, the cache's write and read, and the attention that reads it. What each computes in plain torch, the
library's calls beside it, and the work of one pass.

A case is a dict of plain values. Its "op" is one of

* "norm":       y = rotation of w * x / sqrt(mean(x^2) + eps), for every query and key head;
* "norm_train": the same, then dx, dwq, dwk from dy;
* "write":      new keys and values into the pages of an e4m3 cache, with a scale for each page and head;
* "read":       pages of the cache back to packed bf16 rows;
* "attn":       attention of the last few tokens of every sequence over its cache: O and the rows' log-sum-exp.
"""
import math

import torch

own = False

BF16, F32, F8, I32 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int32


# ---------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------
def _norm(name, op, T, q_heads, k_heads, d, sections, base, interleaved, per_axis, first):
    return {"name": name, "op": op, "T": T, "q_heads": q_heads, "k_heads": k_heads, "d": d, "sections": sections,
            "base": base, "interleaved": interleaved, "per_axis": per_axis, "first": first}


def _cache(name, op, new, start, kv_heads, d, page):
    return {"name": name, "op": op, "new": new, "start": start, "kv_heads": kv_heads, "d": d, "page": page}


def _attn(name, new, lens, heads, kv_heads, d, page, causal):
    return {"name": name, "op": "attn", "new": new, "lens": lens, "heads": heads, "kv_heads": kv_heads, "d": d,
            "page": page, "causal": causal}


def _text(values):
    return ",".join(str(int(x)) for x in values)


def listed():
    return [
        # The next token of five conversations in flight, far into them: latency alone.
        _norm("norm_five_tokens", "norm", 5, 16, 4, 96, "48", 10000.0, False, False, 100003),
        # A long prompt's queries and keys, eight query heads to a key head.
        _norm("norm_prompt", "norm", 28350, 32, 4, 128, "64", 1000000.0, False, False, 0),
        # A training step's short micro-batch of image patches: rows and columns with spectra of their own,
        # neighbouring elements as pairs, heads of 72 of which 8 elements stay unrotated.
        _norm("norm_train_image", "norm_train", 1111, 24, 8, 72, "16,16", 100.0, True, True, 0),
        # A training step of 16,384 tokens at the 1.2B layer's heads, key heads shared.
        _norm("norm_train_long", "norm_train", 16384, 16, 4, 96, "48", 10000.0, False, False, 0),
        # The next token of 77 conversations into part-filled pages.
        _cache("write_77_tokens", "write", _text([1] * 77), _text([17 + 53 * i for i in range(77)]), 8, 128, 64),
        # Packed prompts of uneven length, two of them continuing a page; one sequence brings nothing.
        _cache("write_prompts", "write", "2311,97,1024,0,803,4096,416,7492,123", "0,2048,0,512,0,0,33,0,900", 8, 96, 32),
        # The cached prefix of three short conversations, for the attention of a whole new prompt.
        _cache("read_short", "read", "700,33,1500", "0,0,0", 4, 64, 16),
        # Long documents read back whole.
        _cache("read_documents", "read", "40000,1,25011,4097,33333", "0,0,0,0,0", 8, 128, 64),
        # One conversation 131,071 tokens long with two key heads: the work is split over the cache's length.
        _attn("attn_one_long", "1", "131071", 16, 2, 128, 64, True),
        # The next token of 77 conversations of uneven length, at the 1.2B layer's heads.
        _attn("attn_77_tokens", _text([1] * 77), _text([1 + 29 * i for i in range(77)]), 16, 4, 96, 32, True),
        # A large batch in full flight: 128 conversations, up to 8192 tokens each.
        _attn("attn_128_long", _text([1] * 128), _text([8192 - (i * 2657) % 5003 for i in range(128)]), 64, 8, 128,
              128, True),
        # Drafts of up to six tokens checked at once, in small pages; one conversation has just begun.
        _attn("attn_drafts", "4,6,1,5,4,4,3,6", "1000,3,40,2500,0,517,1800,64", 16, 4, 64, 16, True),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_norm(rng):
    kv = rng.choice([1, 2, 4, 5, 8])
    d = rng.choice([64, 72, 80, 96, 128, 256])
    pairs = d // 2 - rng.choice([0, 0, 4, 8, d // 4])  # some heads keep a part unrotated
    pairs -= pairs % 4
    a = rng.randrange(0, pairs + 1)
    b = rng.randrange(0, pairs - a + 1)
    T = _spread(rng, 1, 16384)
    if rng.random() < 0.5:
        sections = str(pairs)
    else:
        sections = "%d,%d,%d" % (a, b, pairs - a - b)
    q_heads = kv * rng.choice([1, 2, 3, 4])
    while T * (q_heads + kv) * d > 5e7:
        T //= 2
    return {"op": rng.choice(["norm", "norm_train"]), "T": T, "q_heads": q_heads, "k_heads": kv, "d": d,
            "sections": sections, "base": rng.choice([100.0, 10000.0, 1000000.0]), "interleaved": rng.random() < 0.5,
            "per_axis": rng.random() < 0.5, "first": rng.choice([0, 0, 77, 100003, 4000037])}


def _draw_cache(rng):
    G, d, page = rng.choice([1, 2, 4, 5, 8]), rng.choice([64, 80, 96, 128]), rng.choice([16, 32, 64, 128])
    op = rng.choice(["write", "read"])
    if rng.random() < 0.4:  # single tokens
        new = [1] * _spread(rng, 1, 400)
    else:
        T = _spread(rng, 8, 30000)
        parts = [rng.choice([0.0, rng.random(), rng.random(), 1.0]) for _ in range(rng.choice([1, 2, 3, 5, 8, 13]))]
        new = [int(T * x / max(sum(parts), 1.0)) for x in parts]
        new[0] += 1
    start = [rng.choice([0, page * rng.randrange(0, 9), rng.randrange(0, 1500)]) for _ in new]
    return {"op": op, "new": _text(new), "start": _text(start), "kv_heads": G, "d": d, "page": page}


def _draw_attn(rng):
    G = rng.choice([1, 2, 4, 5, 8])
    heads, d, page = G * rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 96, 128]), rng.choice([16, 32, 64, 128])
    most = _spread(rng, 1, 100000)
    n = _spread(rng, 1, max(1, min(256, 2000000 // (most * G))))
    lens = [rng.choice([most, rng.randrange(0, most + 1), rng.randrange(0, most + 1)]) for _ in range(n)]
    lens[0] = most
    new = [1] * n
    if rng.random() < 0.4:  # a few tokens of each; some sequences bring none
        new = [rng.randrange(0, 9) for _ in range(n)]
        new[0] += 1
    return {"op": "attn", "new": _text(new), "lens": _text(lens), "heads": heads, "kv_heads": G, "d": d, "page": page,
            "causal": rng.random() < 0.8}


def draw(rng):
    return rng.choice([_draw_norm, _draw_cache, _draw_attn])(rng)


# ---------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------
def _ints(text):
    return [int(x) for x in text.split(",")]


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _pool(gen, lens, G, d, page):
    """A pool of pages for sequences of these lengths, in an order of its own, with a few pages of nobody. Keys and
    values of a page lie side by side, normal values at scales of their own."""
    counts = [max(1, -(-n // page)) for n in lens]
    used, most = sum(counts), max(counts)
    pages = used + 5
    order = torch.randperm(pages, generator=gen, device="cuda").to(I32)
    at = torch.tensor(_cu(counts), device="cuda")
    col = torch.arange(most, device="cuda")
    idx = torch.minimum(at[:-1, None] + col, at[1:, None] - 1)
    table = order[idx].contiguous()  # behind a sequence's pages: its last page again
    codes = torch.empty(pages, 2, G, page, d, device="cuda", dtype=F8)
    grow = torch.randint(-1, 2, (pages, 2, G), generator=gen, device="cuda").float()
    scales = torch.exp2(grow - 6.0)
    step = max(1, (1 << 26) // (2 * G * page * d))
    for p in range(0, pages, step):  # in pieces: the pool may be much of the card's memory in 32 bits
        part = codes[p:p + step]
        x = torch.randn(part.shape, generator=gen, device="cuda")
        part.copy_((x / scales[p:p + step, ..., None, None]).clamp(-448.0, 448.0))
    return {"kc": codes[:, 0], "vc": codes[:, 1], "ks": scales[:, 0], "vs": scales[:, 1], "table": table}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, device="cuda", generator=gen) * std).to(BF16)

    def empty(*shape, dtype=BF16):
        return torch.empty(*shape, device="cuda", dtype=dtype)

    def ints(values):
        return torch.tensor(values, device="cuda", dtype=I32)

    s = {"case": case}
    if case["op"] in ("norm", "norm_train"):
        T, H, G, d = case["T"], case["q_heads"], case["k_heads"], case["d"]
        # Queries and keys lie in the projection's packed rows, before the values; tokens differ in size.
        s["qkv"] = (normal(T, H + 2 * G, d) * torch.exp(torch.randn(T, 1, 1, device="cuda", generator=gen))).to(BF16)
        s["x"] = s["qkv"][:, :H + G]
        s["y"] = empty(T, H + G, d)
        s["wq"], s["wk"] = ((1.0 + 0.2 * torch.randn(d, device="cuda", generator=gen)).to(BF16) for _ in range(2))
        s["sections"] = tuple(_ints(case["sections"]))
        at = torch.arange(T, device="cuda", dtype=torch.int64)
        side = max(1, int(math.sqrt(T)))
        pos = [at] if len(s["sections"]) == 1 else [at // side, at % side, at % 7][:len(s["sections"])]
        s["pos"] = (torch.stack(pos) + case["first"]).to(I32)
        if case["op"] == "norm_train":
            s["dqkv"] = normal(T, H + 2 * G, d)
            s["dy"], s["dx"] = s["dqkv"][:, :H + G], empty(T, H + G, d)
            s["dwq"], s["dwk"] = empty(d, dtype=F32), empty(d, dtype=F32)
            # Room for any split of the sums over tokens that a library may choose.
            s["sums"] = empty(1024 * 2 * d, dtype=F32).view(torch.uint8)
    elif case["op"] in ("write", "read"):
        new, start = _ints(case["new"]), _ints(case["start"])
        T, G, d = sum(new), case["kv_heads"], case["d"]
        s.update(_pool(gen, [a + b for a, b in zip(new, start)], G, d, case["page"]))
        s["cu"], s["start"], s["max_n"] = ints(_cu(new)), ints(start), max(new)
        if case["op"] == "write":  # keys and values lie in the packed rows of one projection; tokens differ in size
            x = normal(T, 2 * G, d) * torch.exp(0.5 * torch.randn(T, 1, 1, device="cuda", generator=gen))
            s["kv"] = x.to(BF16)
            s["K"], s["V"] = s["kv"][:, :G], s["kv"][:, G:]
        else:
            s["K"], s["V"] = empty(T, G, d), empty(T, G, d)
    else:
        new, lens = _ints(case["new"]), _ints(case["lens"])
        T, H, G, d = sum(new), case["heads"], case["kv_heads"], case["d"]
        s.update(_pool(gen, lens, G, d, case["page"]))
        s["cu"], s["lens"], s["max_q"], s["max_k"] = ints(_cu(new)), ints(lens), max(new), max(lens)
        s["Q"], s["O"], s["LSE"] = normal(T, H, d), empty(T, H, d), empty(H, T, dtype=F32)
        # A workspace for the joins of a split cache, zeroed once.
        s["joins"] = torch.zeros(64 << 20, device="cuda", dtype=torch.uint8)
        s["scale"] = 1.0 / math.sqrt(d)
    return s


# ---------------------------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------------------------
def _angles(s):
    """Cosines and sines [T, 1, pairs]; angles in 64 bits, for far positions."""
    c, pos = s["case"], s["pos"]
    sec = torch.tensor(s["sections"], device=pos.device)
    n = int(sum(s["sections"]))
    axis = torch.repeat_interleave(torch.arange(len(s["sections"]), device=pos.device), sec)
    i = torch.arange(n, device=pos.device, dtype=torch.float64)
    if c["per_axis"]:  # every axis runs through a spectrum of its own
        e = (i - (torch.cumsum(sec, 0) - sec)[axis]) / sec[axis]
    else:
        e = i / n
    ang = pos.to(torch.float64)[axis].t() * torch.exp(-math.log(c["base"]) * e)
    return torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None], n


def _turn(z, cos, sin, n, interleaved):
    out = z.clone()
    if interleaved:
        a, b = z[..., 0:2 * n:2], z[..., 1:2 * n:2]
        out[..., 0:2 * n:2], out[..., 1:2 * n:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = z[..., :n], z[..., n:2 * n]
        out[..., :n], out[..., n:2 * n] = a * cos - b * sin, b * cos + a * sin
    return out


EPS = 1e-6


def _plain_norm(s):
    c = s["case"]
    H = c["q_heads"]
    cos, sin, n = _angles(s)
    x = s["x"].float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    nx = x * r
    is_q = (torch.arange(x.shape[1], device=x.device) < H)[:, None]
    w = torch.where(is_q, s["wq"].float(), s["wk"].float())
    y = _turn(nx * w, cos, sin, n, c["interleaved"]).to(BF16)
    if c["op"] == "norm":
        return y
    g = _turn(s["dy"].float(), cos, -sin, n, c["interleaved"])
    dw = (g * nx).sum(0)
    gw = g * w
    dx = (r * (gw - nx * (gw * nx).mean(-1, keepdim=True))).to(BF16)
    return {"y": y, "dx": dx, "dwq": dw[:H].sum(0), "dwk": dw[H:].sum(0)}


def _owners(cu, T):
    """The sequence of each packed row, and the row's place in it."""
    row = torch.arange(T, device=cu.device)
    seq = torch.bucketize(row, cu[1:].long(), right=True)
    return seq, row - cu.long()[seq]


def _write_one(x, codes, scales, s, page):
    seq, place = _owners(s["cu"], x.shape[0])
    start, n = s["start"].long(), (s["cu"][1:] - s["cu"][:-1]).long()
    at = start[seq] + place
    pg, slot = s["table"][seq, at // page].long(), at % page
    x = x.float()
    G = x.shape[1]
    most = torch.zeros(codes.shape[0], G, device=x.device)
    most.scatter_reduce_(0, pg[:, None].expand(-1, G), x.abs().amax(-1), "amax")
    m, e = torch.frexp(most)  # 448 = 0.875 * 2^9
    e = torch.where(most > 0, e - 9 + (m > 0.875).to(e.dtype), -100).clamp(min=-100)
    need = torch.exp2(e.float())
    # Rows that a sequence's first page holds already: re-rounded where its scale grows.
    p0 = s["table"][torch.arange(n.numel(), device=n.device), torch.minimum(start, (start + n - 1).clamp(min=0)) // page]
    p0 = p0.long()
    held = torch.where(n > 0, start % page, 0)
    before = scales[p0]
    after = torch.where(held[:, None] > 0, torch.maximum(before, need[p0]), before)
    raw = codes.view(torch.uint8)
    first = raw[p0]
    moved = (first.view(F8).float() * (before / after)[..., None, None]).to(F8).view(torch.uint8)
    old = torch.arange(page, device=n.device) < held[:, None]
    raw[p0] = torch.where(old[:, None, :, None], moved, first)
    scales[pg] = need[pg]
    scales[p0] = torch.where(held[:, None] > 0, after, scales[p0])
    raw[pg, :, slot] = (x / scales[pg][..., None]).to(F8).view(torch.uint8)


def _plain_write(s):
    page = s["case"]["page"]
    _write_one(s["K"], s["kc"], s["ks"], s, page)
    _write_one(s["V"], s["vc"], s["vs"], s, page)
    return {"kc": s["kc"], "vc": s["vc"], "ks": s["ks"], "vs": s["vs"]}


def _read_one(codes, scales, s, T, page):
    seq, place = _owners(s["cu"], T)
    at = s["start"].long()[seq] + place
    pg = s["table"][seq, at // page].long()
    rows = codes.view(torch.uint8)[pg, :, at % page].view(F8).float()
    return (rows * scales[pg][..., None]).to(BF16)


def _plain_read(s):
    page, T = s["case"]["page"], s["K"].shape[0]
    return {"K": _read_one(s["kc"], s["ks"], s, T, page), "V": _read_one(s["vc"], s["vs"], s, T, page)}


def _whole(codes, scales, table):
    """The cache of every sequence side by side, [sequences, heads, 1, tokens, d]."""
    t = table.long()
    x = codes.view(torch.uint8)[t].view(F8).float() * scales[t][..., None, None]  # [sequences, pages, heads, page, d]
    return x.transpose(1, 2).flatten(2, 3)[:, :, None]


def _plain_attn(s):
    c = s["case"]
    H, G, d, T = c["heads"], c["kv_heads"], c["d"], s["Q"].shape[0]
    dev, N, mq = s["Q"].device, s["lens"].numel(), s["max_q"]
    n, lens = (s["cu"][1:] - s["cu"][:-1]).long(), s["lens"].long()
    # Queries padded to the longest sequence's: [sequences, kv heads, group, queries, d].
    iq = torch.arange(mq, device=dev)
    real = iq < n[:, None]
    at = (s["cu"][:-1].long()[:, None] + iq).clamp(max=max(T - 1, 0))
    q = s["Q"][at].float().view(N, mq, G, H // G, d).permute(0, 2, 3, 1, 4)
    k = _whole(s["kc"], s["ks"], s["table"])
    ik = torch.arange(k.shape[3], device=dev)
    see = ik < lens[:, None, None]
    if c["causal"]:  # the last query sees the last key
        see = see & (ik <= (iq + (lens - n)[:, None])[..., None])
    see = see[:, None, None]
    sc = torch.matmul(q, k.transpose(-1, -2)) * s["scale"]
    del k
    sc = torch.where(see, sc, -math.inf)
    m = sc.amax(-1, keepdim=True)
    m = torch.where(m > -math.inf, m, 0.0)
    p = torch.exp(sc - m)
    del sc
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, _whole(s["vc"], s["vs"], s["table"])) / torch.where(l > 0, l, 1.0)
    lse = (m + torch.log(l)).squeeze(-1)  # -inf where nothing is seen
    seq, place = _owners(s["cu"], T)
    O = o.flatten(1, 2)[seq, :, place].to(BF16)
    return {"O": O, "LSE": lse.flatten(1, 2)[seq, :, place].t().contiguous()}


# ---------------------------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------------------------
def _own(s):
    import tensor_transformer_layer_gb300 as mp

    c = s["case"]
    if c["op"] in ("norm", "norm_train"):
        how = dict(q_heads=c["q_heads"], sections=s["sections"], base=c["base"], eps=EPS, interleaved=c["interleaved"],
                   per_axis=c["per_axis"])
        mp.mp_qk_norm_rope(s["x"], s["y"], s["wq"], s["wk"], s["pos"], **how)
        if c["op"] == "norm":
            return s["y"]
        mp.mp_qk_norm_rope_bwd(s["x"], s["dy"], s["dx"], s["wq"], s["wk"], s["dwq"], s["dwk"], s["pos"], s["sums"], **how)
        return {"y": s["y"], "dx": s["dx"], "dwq": s["dwq"], "dwk": s["dwk"]}
    if c["op"] == "write":
        mp.mp_kv_cache_write(s["K"], s["V"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["cu"], s["start"],
                             max_n=s["max_n"])
        return {"kc": s["kc"], "vc": s["vc"], "ks": s["ks"], "vs": s["vs"]}
    if c["op"] == "read":
        mp.mp_kv_cache_read(s["kc"], s["vc"], s["ks"], s["vs"], s["K"], s["V"], s["table"], s["cu"], s["start"],
                            max_n=s["max_n"])
        return {"K": s["K"], "V": s["V"]}
    mp.mp_attn_cache_fwd(s["Q"], s["kc"], s["vc"], s["ks"], s["vs"], s["O"], s["LSE"], s["table"], s["cu"], s["lens"],
                         s["joins"], max_q=s["max_q"], causal=c["causal"], scale=s["scale"])
    return {"O": s["O"], "LSE": s["LSE"]}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op in ("norm", "norm_train"):
        return _plain_norm(state)
    if op == "write":
        return _plain_write(state)
    return _plain_read(state) if op == "read" else _plain_attn(state)


# ---------------------------------------------------------------------------------------------
# Work
# ---------------------------------------------------------------------------------------------
def work(case):
    if case["op"] in ("norm", "norm_train"):
        n = case["T"] * (case["q_heads"] + case["k_heads"]) * case["d"]
        axes = len(_ints(case["sections"]))
        if case["op"] == "norm":
            return {"bytes": 4 * n + 4 * axes * case["T"] + 4 * case["d"], "flops": 9 * n}
        # x is read by both directions; dy in, dx out
        return {"bytes": 10 * n + 8 * axes * case["T"] + 16 * case["d"], "flops": 25 * n}
    if case["op"] in ("write", "read"):
        new, start, G, d, page = _ints(case["new"]), _ints(case["start"]), case["kv_heads"], case["d"], case["page"]
        pages = sum(-(-(a + b) // page) - b // page for a, b in zip(new, start) if a)
        n = 2 * sum(new) * G * d
        return {"bytes": 3 * n + 8 * G * pages + 4 * pages + 8 * len(new), "flops": 2 * n}
    new, lens, H, G, d = _ints(case["new"]), _ints(case["lens"]), case["heads"], case["kv_heads"], case["d"]
    T, keys, pairs = sum(new), 0, 0
    for nq, nk in zip(new, lens):
        if nq:
            keys += nk
            pairs += sum(max(0, nk - nq + i + 1) for i in range(nq)) if case["causal"] else nq * nk
    pages = sum(-(-nk // case["page"]) for nq, nk in zip(new, lens) if nq)
    return {"bytes": 2 * keys * G * d + 8 * pages * G + 4 * pages + 4 * T * H * d + 4 * T * H, "flops": 4 * H * pairs * d}


# ---------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------------------------
def _exact_rotation(x, case, pos, back):
    n = sum(_ints(case["sections"]))
    out = torch.empty_like(x).copy_(x)
    pair = 0
    for axis, size in enumerate(_ints(case["sections"])):
        for j in range(size):
            theta = pos[axis].double() * case["base"] ** -(j / size if case["per_axis"] else pair / n)
            turn = torch.polar(torch.ones_like(theta), -theta if back else theta)[:, None]
            ia, ib = (2 * pair, 2 * pair + 1) if case["interleaved"] else (pair, pair + n)
            z = torch.complex(x[..., ia], x[..., ib]) * turn
            out[..., ia], out[..., ib] = z.real, z.imag
            pair += 1
    return out


def _exact_norm(case, s):
    H, train = case["q_heads"], case["op"] == "norm_train"
    x, wq, wk = (s[k].double().requires_grad_(train) for k in ("x", "wq", "wk"))
    w = torch.cat([wq.expand(H, -1), wk.expand(x.shape[1] - H, -1)])
    z = x / torch.linalg.vector_norm(x, dim=-1, keepdim=True).square().div(case["d"]).add(EPS).sqrt() * w
    y = _exact_rotation(z.detach(), case, s["pos"], False)
    if not train:
        return y
    g = _exact_rotation(s["dy"].double(), case, s["pos"], True)
    dx, dwq, dwk = torch.autograd.grad(z, (x, wq, wk), g)
    return {"y": y, "dx": dx, "dwq": dwq, "dwk": dwk}


def _e4m3_values():
    """The 127 finite values from 0 to 448, by code."""
    return [m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)][:127]


def _nearest(x):
    """x rounded to e4m3 (ties to the even code), in 64 bits."""
    v = torch.tensor(_e4m3_values(), device=x.device, dtype=torch.float64)
    mid = (v[1:] + v[:-1]) / 2
    a = x.abs()
    i = torch.searchsorted(mid, a)  # a <= mid[i]
    tie = (i < 126) & (a == mid[i.clamp(max=125)]) & (i % 2 == 1)
    return torch.copysign(v[i + tie.long()], x)


def _exact_write(case, s):
    page, new, start = case["page"], _ints(case["new"]), _ints(case["start"])
    out = {}
    for x, codes, scales, kc, ks in (("K", "kc", "ks", "kc", "ks"), ("V", "vc", "vs", "vc", "vs")):
        c, sc, table = s[codes].double(), s[scales].double().clone(), s["table"].tolist()
        row = 0
        for i, n in enumerate(new):
            left, at = n, start[i]
            while left:
                pg, a = table[i][at // page], at % page
                b = min(page, a + left)
                part = s[x][row:row + b - a].double().transpose(0, 1)  # [heads, rows, d]
                most = part.abs().amax((1, 2))
                need = torch.full_like(most, 2.0 ** -100)
                e = torch.ceil(torch.log2(most / 448.0)).clamp(min=-100)
                e = torch.where(448.0 * torch.exp2(e - 1) >= most, e - 1, e).clamp(min=-100)
                e = torch.where(448.0 * torch.exp2(e) < most, e + 1, e)
                need = torch.where(most > 0, torch.exp2(e), need)
                scale = torch.maximum(need, sc[pg]) if a else need
                if a:
                    c[pg, :, :a] = _nearest(c[pg, :, :a] * (sc[pg] / scale)[:, None, None])
                c[pg, :, a:b] = _nearest(part / scale[:, None, None])
                sc[pg] = scale
                row, left, at = row + b - a, left - (b - a), at + b - a
        out[kc], out[ks] = c, sc
    return out


def _exact_rows(s, codes, scales, i, first, count, page):
    """`count` rows of sequence i's cache from `first` on, [rows, heads, d]."""
    if count == 0:
        return s[codes].new_zeros((0,) + (s[codes].shape[1], s[codes].shape[3]), dtype=torch.float64)
    lo, hi = first // page, -(-(first + count) // page)
    ids = s["table"][i, lo:hi].long()
    x = s[codes].view(torch.uint8)[ids].view(F8).double() * s[scales][ids].double()[..., None, None]
    return x.transpose(1, 2).reshape(-1, x.shape[1], x.shape[3])[first - lo * page:][:count]


def _exact_read(case, s):
    todo = list(enumerate(zip(_ints(case["start"]), _ints(case["new"]))))
    return {k: torch.cat([_exact_rows(s, c, z, i, a, n, case["page"]) for i, (a, n) in todo])
            for k, c, z in (("K", "kc", "ks"), ("V", "vc", "vs"))}


def _exact_attn(case, s):
    H, G, d = case["heads"], case["kv_heads"], case["d"]
    Q = s["Q"].double()
    res = {"O": torch.zeros_like(Q), "LSE": Q.new_full((H, Q.shape[0]), -math.inf)}
    row = 0
    for i, (nq, nk) in enumerate(zip(_ints(case["new"]), _ints(case["lens"]))):
        rows = slice(row, row + nq)
        row += nq
        if nq == 0 or nk == 0:
            continue
        k, v = (_exact_rows(s, a, b, i, 0, nk, case["page"]).transpose(0, 1) for a, b in (("kc", "ks"), ("vc", "vs")))
        hidden = torch.zeros(nq, nk, device=Q.device, dtype=torch.bool)
        if case["causal"]:
            hidden = torch.ones_like(hidden).triu(nk - nq + 1)
        live = ~hidden.all(1)
        q = Q[rows][live].view(-1, G, H // G, d).permute(1, 2, 0, 3)  # [G, group, queries, d]
        z = torch.einsum("grqd,gkd->grqk", q, k) / math.sqrt(d)
        z = z.masked_fill(hidden[live], -math.inf)
        o = torch.einsum("grqk,gkd->qgrd", torch.softmax(z, -1), v).flatten(1, 2)
        at = torch.arange(rows.start, rows.stop, device=Q.device)[live]
        res["O"][at] = o
        res["LSE"][:, at] = torch.logsumexp(z, -1).flatten(0, 1)
    return res


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm", "norm_train"):
        return _exact_norm(case, s)
    if case["op"] == "write":
        return _exact_write(case, s)
    return _exact_read(case, s) if case["op"] == "read" else _exact_attn(case, s)
