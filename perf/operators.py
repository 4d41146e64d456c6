"""Measured cases of the transformer layer's position rotation, packed attention and gated feed-forward
operators: what each computes in plain torch, the library's calls beside it, and the work of one pass.

A case is a dict of plain values. Its "op" is one of

* "rope":       y = rotation of every head of x by the angles of several position axes (or back, for gradients);
* "attn":       attention over packed sequences, forward only: O and the rows' log-sum-exp;
* "attn_train": the same forward, then dQ, dK, dV from dO;
* "glu":        Y = act(X Wg) * (X Wu), Z = Y Wd, forward only;
* "glu_train":  the same forward, then dX, dW = [dWg | dWu], dWd from dZ.
"""
import math

import torch

own = False

BF16 = torch.bfloat16


# ---------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------
def _rope(name, grid, heads, kv_heads, d, sections, base, interleaved, per_axis, inverse, first):
    return {"name": name, "op": "rope", "grid": grid, "heads": heads, "kv_heads": kv_heads, "d": d,
            "sections": sections, "base": base, "interleaved": interleaved, "per_axis": per_axis,
            "inverse": inverse, "first": first}


def _attn(name, op, q_lens, k_lens, heads, kv_heads, d, causal):
    return {"name": name, "op": op, "q_lens": q_lens, "k_lens": k_lens, "heads": heads, "kv_heads": kv_heads,
            "d": d, "causal": causal}


def _glu(name, op, T, h, f, t, act):
    return {"name": name, "op": op, "T": T, "h": h, "f": f, "t": t, "act": act}


def listed():
    return [
        # One new token of each of five conversations in flight, far into them: latency alone.
        _rope("rope_five_tokens", "5,1,1", 16, 16, 96, "16,16,16", 10000.0, False, False, False, 100003),
        # A video clip of 21 frames of 30 x 45 patches, queries and keys of the 2.5B layer's heads.
        _rope("rope_video", "21,30,45", 20, 20, 96, "16,16,16", 10000.0, False, False, False, 0),
        # The gradient of an image batch's rotation: rows and columns with spectra of their own, neighbouring
        # elements as pairs, fewer key heads than query heads, heads of 72.
        _rope("rope_image_grad", "9,51,67", 24, 8, 72, "0,18,18", 100.0, True, True, True, 0),
        # A few short sequences, one of them a single token: latency.
        _attn("attn_train_short", "attn_train", "1,17,64,130", "1,17,64,130", 4, 4, 64, True),
        # Documents of uneven length packed into one batch of 8192 tokens, heads of the 1.2B layer, key heads shared.
        _attn("attn_train_packed", "attn_train", "2311,97,1024,1,803,2048,416,1492", "2311,97,1024,1,803,2048,416,1492",
              16, 4, 96, True),
        # One long document, eight query heads on two key heads.
        _attn("attn_train_long", "attn_train", "16384", "16384", 8, 2, 128, True),
        # Two clips whose patches all see each other, and a text of another length that they read.
        _attn("attn_train_clips", "attn_train", "3510,1755", "4022,1801", 24, 24, 64, False),
        # The forward alone, as in evaluation: four prompts of which some continue a longer prefix; one row of the
        # last sequence sees no key at all.
        _attn("attn_prefix", "attn", "512,700,33,1025", "2048,700,1500,1024", 20, 20, 96, True),
        # One token through the 1.2B layer's width.
        _glu("glu_one_token", "glu", 1, 1536, 4096, 8, "silu"),
        # A batch of 77 tokens, one from each conversation in flight, through the 4.2B layer's width.
        _glu("glu_77_tokens", "glu", 77, 2304, 6144, 8, "silu"),
        # A training step of an uneven micro-batch with the GeLU gate.
        _glu("glu_train_uneven", "glu_train", 1111, 1920, 5120, 4, "gelu"),
        # A training step of the 4.2B layer's width.
        _glu("glu_train", "glu_train", 8192, 2304, 6144, 8, "silu"),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng):
    kv = rng.choice([1, 2, 4, 5, 8])
    return kv * rng.choice([1, 2, 3, 4]), kv


def _draw_rope(rng):
    heads, kv = _heads(rng)
    d = rng.choice([64, 72, 80, 96, 128])
    pairs = d // 2 - rng.choice([0, 0, 4, 8])  # some heads keep a part unrotated
    pairs -= pairs % 4
    a = rng.randrange(0, pairs + 1)
    b = rng.randrange(0, pairs - a + 1)
    T = _spread(rng, 1, 30000)
    rows = max(1, int(round(T ** 0.33)))
    cols = max(1, int(round((T / rows) ** 0.5)))
    frames = max(1, T // (rows * cols))
    return {"op": "rope", "grid": "%d,%d,%d" % (frames, rows, cols), "heads": heads, "kv_heads": kv, "d": d,
            "sections": "%d,%d,%d" % (a, b, pairs - a - b), "base": rng.choice([100.0, 10000.0, 1000000.0]),
            "interleaved": rng.random() < 0.5, "per_axis": rng.random() < 0.5, "inverse": rng.random() < 0.5,
            "first": rng.choice([0, 0, 77, 100003, 4000037])}


def _draw_attn(rng):
    heads, kv = _heads(rng)
    d, causal, op = rng.choice([64, 96, 128]), rng.random() < 0.7, rng.choice(["attn", "attn_train", "attn_train"])
    T = _spread(rng, 1 if op == "attn" else 16, min(8192, int((1.9e12 / (14 * heads * d)) ** 0.5)))
    n = min(T, rng.choice([1, 1, 2, 3, 5, 8, 13]))
    parts = [rng.choice([0.0, rng.random(), rng.random(), 1.0]) for _ in range(n)]
    q = [int(T * x / max(sum(parts), 1.0)) for x in parts]  # some of them empty
    q[0] += 1 if sum(q) == 0 else 0
    k = list(q)
    if rng.random() < 0.4:  # keys of another length: a prefix, another sequence, none at all
        k = [max(0, x + rng.choice([0, 1, -1, rng.randrange(0, 300), -rng.randrange(0, 300)])) for x in q]
    if sum(k) == 0 or op == "attn_train" and sum(_seen(a, b, causal) for a, b in zip(q, k)) < 4 * sum(q):
        q, k = [T], [T]  # rows of one key have no gradient for queries and keys but rounding
    return {"op": op, "q_lens": ",".join(map(str, q)),
            "k_lens": ",".join(map(str, k)), "heads": heads, "kv_heads": kv, "d": d,
            "causal": causal}


def _draw_glu(rng):
    t = rng.choice([1, 2, 4, 8])
    h = 64 * _spread(rng, 4, 36)
    f = 64 * t * max(1, _spread(rng, 8, 96) // t)
    train = rng.random() < 0.6
    return {"op": "glu_train" if train else "glu", "T": _spread(rng, 1, 8192 if train else 4096), "h": h, "f": f,
            "t": t, "act": rng.choice(["silu", "gelu"])}


def draw(rng):
    return rng.choice([_draw_rope, _draw_attn, _draw_glu])(rng)


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


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, device="cuda", generator=gen) * std).to(BF16)

    def empty(*shape, dtype=BF16):
        return torch.empty(*shape, device="cuda", dtype=dtype)

    s = {"case": case}
    if case["op"] == "rope":
        grid = _ints(case["grid"])
        T = grid[0] * grid[1] * grid[2]
        nh = case["heads"] + case["kv_heads"]
        # Queries and keys lie in the projection's packed rows, before the values.
        s["qkv"] = normal(T, nh + case["kv_heads"], case["d"])
        s["x"] = s["qkv"][:, :nh]
        s["y"] = empty(T, nh, case["d"])
        at = torch.arange(T, device="cuda", dtype=torch.int64)
        pos = torch.stack([at // (grid[1] * grid[2]), at // grid[2] % grid[1], at % grid[2]])
        s["pos"] = (pos + case["first"]).to(torch.int32)
        s["sections"] = tuple(_ints(case["sections"]))
    elif case["op"] in ("attn", "attn_train"):
        ql, kl = _ints(case["q_lens"]), _ints(case["k_lens"])
        Tq, Tk, H, G, d = sum(ql), sum(kl), case["heads"], case["kv_heads"], case["d"]
        s["Q"], s["O"] = normal(Tq, H, d), empty(Tq, H, d)
        s["LSE"] = empty(H, Tq, dtype=torch.float32)
        if ql == kl:  # keys and values lie in the packed rows of one projection
            s["kv"] = normal(Tk, 2 * G, d)
            s["K"], s["V"] = s["kv"][:, :G], s["kv"][:, G:]
        else:
            s["K"], s["V"] = normal(Tk, G, d), normal(Tk, G, d)
        s["cu_q"] = torch.tensor(_cu(ql), device="cuda", dtype=torch.int32)
        s["cu_k"] = torch.tensor(_cu(kl), device="cuda", dtype=torch.int32)
        s["max_q"], s["max_k"] = max(ql), max(kl)
        s["scale"] = 1.0 / math.sqrt(d)
        if case["op"] == "attn_train":
            s["dO"] = normal(Tq, H, d)
            s["dQ"], s["dK"], s["dV"] = empty(Tq, H, d), empty(Tk, G, d), empty(Tk, G, d)
            s["delta"] = empty(H, Tq, dtype=torch.float32)
    else:
        T, h, f = case["T"], case["h"], case["f"]
        s["X"], s["W"], s["Wd"] = normal(T, h), normal(h, 2 * f, std=0.02), normal(f, h, std=0.02)
        s["Z"], s["Y"] = empty(T, h), empty(T, f)
        if case["op"] == "glu_train":
            s["dZ"] = normal(T, h)
            s["GU"], s["dGU"] = empty(T, 2 * f), empty(T, 2 * f)
            s["dX"], s["dW"], s["dWd"] = empty(T, h), empty(h, 2 * f), empty(f, h)
    return s


# ---------------------------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------------------------
def _plain_rope(s):
    c, x, pos = s["case"], s["x"], s["pos"]
    dev, sec = x.device, torch.tensor(s["sections"], device=x.device)
    n = int(sum(s["sections"]))
    axis = torch.repeat_interleave(torch.arange(len(s["sections"]), device=dev), sec)
    i = torch.arange(n, device=dev, dtype=torch.float64)
    if c["per_axis"]:  # every axis runs through a spectrum of its own
        start = torch.cumsum(sec, 0) - sec
        e = (i - start[axis]) / sec[axis]
    else:
        e = i / max(n, 1)
    freq = torch.exp(-math.log(c["base"]) * e)
    ang = pos.to(torch.float64)[axis].t() * freq  # [T, n]; 64 bits, for far positions
    if c["inverse"]:
        ang = -ang
    cos, sin = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]
    xf = x.float()
    y = xf.clone()
    if c["interleaved"]:
        a, b = xf[..., 0:2 * n:2], xf[..., 1:2 * n:2]
        y[..., 0:2 * n:2], y[..., 1:2 * n:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = xf[..., :n], xf[..., n:2 * n]
        y[..., :n], y[..., n:2 * n] = a * cos - b * sin, b * cos + a * sin
    return y.to(BF16)


def _padded(x, cu, most):
    """Packed rows [T, ...] as [sequences, most, ...] with zeros behind each sequence, and which rows are real."""
    at = torch.arange(most, device=x.device)
    n = (cu[1:] - cu[:-1]).long()
    real = at[None] < n[:, None]
    idx = (cu[:-1].long()[:, None] + at[None]).clamp(max=max(x.shape[0] - 1, 0))
    rows = x[idx].float()
    return torch.where(real.view(real.shape + (1,) * (x.dim() - 1)), rows, 0.0), real


def _plain_attn(s):
    c = s["case"]
    H, G, d = c["heads"], c["kv_heads"], c["d"]
    r = H // G
    q, q_real = _padded(s["Q"], s["cu_q"], s["max_q"])
    k, k_real = _padded(s["K"], s["cu_k"], s["max_k"])
    v, _ = _padded(s["V"], s["cu_k"], s["max_k"])
    N, mq, mk = q.shape[0], q.shape[1], k.shape[1]
    q = q.view(N, mq, G, r, d).permute(0, 2, 3, 1, 4)                # [N, G, r, mq, d]
    k, v = k.permute(0, 2, 1, 3)[:, :, None], v.permute(0, 2, 1, 3)[:, :, None]  # [N, G, 1, mk, d]
    see = q_real[:, :, None] & k_real[:, None]
    if c["causal"]:  # the last query sees the last key
        off = (s["cu_k"][1:] - s["cu_k"][:-1]) - (s["cu_q"][1:] - s["cu_q"][:-1])
        iq, ik = torch.arange(mq, device=q.device), torch.arange(mk, device=q.device)
        see = see & (ik[None, None] <= iq[None, :, None] + off[:, None, None])
    see = see[:, None, None]
    sc = torch.matmul(q, k.transpose(-1, -2)) * s["scale"]
    sc = torch.where(see, sc, -math.inf)
    m = sc.amax(-1, keepdim=True)
    m = torch.where(m > -math.inf, m, 0.0)
    p = torch.exp(sc - m)
    del sc
    l = p.sum(-1, keepdim=True)
    p = p / torch.where(l > 0, l, 1.0)
    lse = (m + torch.log(l)).squeeze(-1)                              # -inf where nothing is seen
    o = torch.matmul(p, v)

    def packed(x, real):                                              # [N, heads.., rows, d] -> [T, heads, d]
        return x.flatten(1, 2).permute(0, 2, 1, 3)[real].to(BF16)

    out = {"O": packed(o, q_real), "LSE": lse.flatten(1, 2).permute(0, 2, 1)[q_real].t().contiguous()}
    if c["op"] == "attn":
        return out
    do, _ = _padded(s["dO"], s["cu_q"], s["max_q"])
    do = do.view(N, mq, G, r, d).permute(0, 2, 3, 1, 4)
    dv = torch.matmul(p.transpose(-1, -2), do).sum(2, keepdim=True)
    ds = torch.matmul(do, v.transpose(-1, -2))
    ds -= (do * o).sum(-1, keepdim=True)
    ds *= p
    dq = torch.matmul(ds, k) * s["scale"]
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(2, keepdim=True) * s["scale"]
    out.update(dQ=packed(dq, q_real), dK=packed(dk, k_real), dV=packed(dv, k_real))
    return out


def _erf_phi(g):
    """Normal distribution function and density."""
    return 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5))), torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2.0 * math.pi))


def _plain_glu(s):
    c = s["case"]
    f = c["f"]
    X, W, Wd = s["X"].float(), s["W"].float(), s["Wd"].float()
    gu = X @ W
    g, u = gu[:, :f], gu[:, f:]
    if c["act"] == "silu":
        sg = 1.0 / (1.0 + torch.exp(-g))
        a, da = g * sg, sg * (1.0 + g * (1.0 - sg))
    else:
        cdf, pdf = _erf_phi(g)
        a, da = g * cdf, cdf + g * pdf
    y = a * u
    Z = y @ Wd
    if c["op"] == "glu":
        return {"Z": Z.to(BF16), "Y": y.to(BF16)}
    dZ = s["dZ"].float()
    dy = dZ @ Wd.t()
    dgu = torch.cat([dy * u * da, dy * a], 1)
    return {"Z": Z.to(BF16), "Y": y.to(BF16), "dX": (dgu @ W.t()).to(BF16), "dW": (X.t() @ dgu).to(BF16),
            "dWd": (y.t() @ dZ).to(BF16)}


# ---------------------------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------------------------
def _own(s):
    import tensor_transformer_layer_gb300 as mp

    c = s["case"]
    if c["op"] == "rope":
        mp.mp_rope_axes(s["x"], s["y"], s["pos"], sections=s["sections"], base=c["base"],
                        interleaved=c["interleaved"], per_axis=c["per_axis"], inverse=c["inverse"])
        return s["y"]
    if c["op"] in ("attn", "attn_train"):
        how = dict(max_q=s["max_q"], max_k=s["max_k"], causal=c["causal"], scale=s["scale"])
        mp.mp_attn_varlen_fwd(s["Q"], s["K"], s["V"], s["O"], s["LSE"], s["cu_q"], s["cu_k"], **how)
        out = {"O": s["O"], "LSE": s["LSE"]}
        if c["op"] == "attn_train":
            mp.mp_attn_varlen_bwd(s["Q"], s["K"], s["V"], s["O"], s["LSE"], s["dO"], s["dQ"], s["dK"], s["dV"],
                                  s["delta"], s["cu_q"], s["cu_k"], **how)
            out.update(dQ=s["dQ"], dK=s["dK"], dV=s["dV"])
        return out
    if c["op"] == "glu":
        mp.mp_glu_fwd(s["X"], s["W"], s["Wd"], s["Z"], s["Y"], None, t=c["t"], act=c["act"])
        return {"Z": s["Z"], "Y": s["Y"]}
    mp.mp_glu_fwd(s["X"], s["W"], s["Wd"], s["Z"], s["Y"], s["GU"], t=c["t"], act=c["act"])
    mp.mp_glu_bwd(s["X"], s["W"], s["Wd"], s["GU"], s["Y"], s["dZ"], s["dX"], s["dW"], s["dWd"], s["dGU"], t=c["t"],
                  act=c["act"])
    return {"Z": s["Z"], "Y": s["Y"], "dX": s["dX"], "dW": s["dW"], "dWd": s["dWd"]}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "rope":
        return _plain_rope(state)
    return _plain_attn(state) if op in ("attn", "attn_train") else _plain_glu(state)


# ---------------------------------------------------------------------------------------------
# Work
# ---------------------------------------------------------------------------------------------
def _seen(nq, nk, causal):
    """Query-key pairs of one sequence."""
    if not causal:
        return nq * nk
    off = nk - nq
    first = max(0, -off)  # rows before it see nothing
    return sum(i + off + 1 for i in range(first, nq))


def work(case):
    if case["op"] == "rope":
        T = math.prod(_ints(case["grid"]))
        n = T * (case["heads"] + case["kv_heads"])
        pairs = sum(_ints(case["sections"]))
        return {"bytes": 2 * 2 * n * case["d"] + 12 * T, "flops": 6 * n * pairs}
    if case["op"] in ("attn", "attn_train"):
        ql, kl = _ints(case["q_lens"]), _ints(case["k_lens"])
        H, G, d = case["heads"], case["kv_heads"], case["d"]
        pairs = H * sum(_seen(a, b, case["causal"]) for a, b in zip(ql, kl))
        q, kv = 2 * sum(ql) * H * d, 2 * sum(kl) * G * d
        n_bytes, flops = 2 * q + 2 * kv + 4 * H * sum(ql), 4 * pairs * d
        if case["op"] == "attn_train":  # dO in; dQ, dK, dV out
            n_bytes, flops = n_bytes + 2 * q + 2 * kv, flops + 10 * pairs * d
        return {"bytes": n_bytes, "flops": flops}
    T, h, f = case["T"], case["h"], case["f"]
    n_bytes, flops = 2 * (2 * T * h + T * f + 3 * h * f), 6 * T * h * f
    if case["op"] == "glu_train":  # dZ in; dX and the weights' gradients out
        n_bytes, flops = n_bytes + 2 * (2 * T * h + 3 * h * f), flops + 12 * T * h * f
    return {"bytes": n_bytes, "flops": flops}


# ---------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------------------------
def _exact_rope(case, s):
    n = sum(_ints(case["sections"]))
    x = s["x"].double()
    z_all = torch.empty_like(x).copy_(x)
    pair, pos = 0, s["pos"].double()
    for axis, size in enumerate(_ints(case["sections"])):
        for j in range(size):
            expo = j / size if case["per_axis"] else pair / n
            theta = pos[axis] * case["base"] ** -expo
            turn = torch.polar(torch.ones_like(theta), -theta if case["inverse"] else theta)[:, None]
            ia, ib = (2 * pair, 2 * pair + 1) if case["interleaved"] else (pair, pair + n)
            z = torch.complex(x[..., ia], x[..., ib]) * turn
            z_all[..., ia], z_all[..., ib] = z.real, z.imag
            pair += 1
    return z_all


def _exact_attn(case, s):
    H, G, d = case["heads"], case["kv_heads"], case["d"]
    train = case["op"] == "attn_train"
    Q, K, V = (s[x].double() for x in ("Q", "K", "V"))
    res = {"O": torch.zeros_like(Q), "LSE": Q.new_full((H, Q.shape[0]), -math.inf)}
    if train:
        res.update(dQ=torch.zeros_like(Q), dK=torch.zeros_like(K), dV=torch.zeros_like(V))
    q0 = k0 = 0
    for nq, nk in zip(_ints(case["q_lens"]), _ints(case["k_lens"])):
        rows, cols = slice(q0, q0 + nq), slice(k0, k0 + nk)
        q0, k0 = q0 + nq, k0 + nk
        if nq == 0 or nk == 0:
            continue
        hidden = torch.zeros(nq, nk, device=Q.device, dtype=torch.bool)
        if case["causal"]:
            hidden = torch.ones_like(hidden).triu(nk - nq + 1)
        live = ~hidden.all(1)
        for head in range(H):
            g = head // (H // G)
            q, k, v = (x.clone().requires_grad_(train) for x in (Q[rows, head], K[cols, g], V[cols, g]))
            z = (q @ k.t() / math.sqrt(d))[live].masked_fill(hidden[live], -math.inf)
            o = torch.softmax(z, -1) @ v
            res["O"][rows, head][live] = o.detach()
            res["LSE"][head, rows][live] = torch.logsumexp(z.detach(), -1)
            if train:
                gq, gk, gv = torch.autograd.grad(o, (q, k, v), s["dO"][rows, head][live].double())
                res["dQ"][rows, head] = gq
                res["dK"][cols, g] += gk
                res["dV"][cols, g] += gv
    return res


def _exact_glu(case, s):
    train = case["op"] == "glu_train"
    X, W, Wd = (s[x].double().requires_grad_(train) for x in ("X", "W", "Wd"))
    gate, up = (X @ W).chunk(2, 1)
    act = torch.nn.functional.silu if case["act"] == "silu" else torch.nn.functional.gelu
    Y = act(gate) * up
    Z = Y @ Wd
    if not train:
        return {"Z": Z, "Y": Y}
    dX, dW, dWd = torch.autograd.grad(Z, (X, W, Wd), s["dZ"].double())
    return {"Z": Z.detach(), "Y": Y.detach(), "dX": dX, "dW": dW, "dWd": dWd}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(case, s)
    return _exact_attn(case, s) if case["op"] in ("attn", "attn_train") else _exact_glu(case, s)
