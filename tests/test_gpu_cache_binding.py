"""The two ways into the entry points of a decoding step, the extension's and the checks' in Python: one answer, one refusal."""
import threading

import pytest
import torch

import tensor_transformer_layer_gb300 as mp
from cache_util import cu_of, ints, page_table, pool

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


class _Recorder:
    """The extension, with the answers of its functions kept."""

    def __init__(self, bind):
        self.bind, self.answers = bind, []

    def __getattr__(self, name):
        f = getattr(self.bind, name)

        def g(*a):
            self.answers.append(f(*a))
            return self.answers[-1]
        return g


class _Off:
    def __getattr__(self, name):
        return lambda *a: None


def _randn(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(BF16).cuda()


class Step:
    """One call of each operator on small inputs; `change` replaces arguments, `out` names the tensors that are compared."""

    def __init__(self, strided=False, T=7):
        heads, kv, d, page = 8, 2, 64, 16
        at_end, new = [T, 33, 0], [T, 2, 0]
        total, most = sum(new), max(new)

        def rows(h, seed):
            return _randn(total, h + (1 if strided else 0), d, seed=seed)[:, :h]

        table, pages = page_table([n + 1 for n in at_end], page, 3)
        codes, scales = pool(pages, kv, page, d, 4)
        codes, scales = codes.cuda(), scales.cuda()
        table, cu = table.cuda(), cu_of(new).cuda()
        start = ints(n - m for n, m in zip(at_end, new)).cuda()
        lens = ints(at_end).cuda()
        pos = torch.arange(total, dtype=torch.int32).expand(2, -1).contiguous().cuda()
        if strided:
            kc, vc, ks, vs = codes[:, 0], codes[:, 1], scales[:, 0], scales[:, 1]
        else:
            kc, vc = codes[:, 0].contiguous(), codes[:, 1].contiguous()
            ks, vs = scales[:, 0].contiguous(), scales[:, 1].contiguous()
        cache = dict(kc=kc, vc=vc, ks=ks, vs=vs, page_table=table)
        rot = dict(q_heads=heads - kv, sections=(16, 16), wq=_randn(d, seed=5), wk=_randn(d, seed=6), pos=pos)
        nan = float("nan")
        f32 = dict(dtype=torch.float32, device="cuda")
        self.calls = {
            "mp_qk_norm_rope": (dict(x=rows(heads, 1), y=rows(heads, 2), **rot), ["y"]),
            "mp_qk_norm_rope_bwd": (dict(x=rows(heads, 1), dy=rows(heads, 2), dx=rows(heads, 3), dwq=torch.full((d,), nan, **f32),
                                         dwk=torch.full((d,), nan, **f32), **rot,
                                         workspace=torch.zeros(mp.mp_qk_norm_rope_bwd_workspace_bytes(total, heads, d),
                                                               dtype=torch.uint8, device="cuda")), ["dx", "dwq", "dwk"]),
            "mp_kv_cache_write": (dict(K=rows(kv, 7), V=rows(kv, 8), **cache, cu=cu, start=start, max_n=most),
                                  ["kc", "vc", "ks", "vs"]),
            "mp_kv_cache_read": (dict(K=rows(kv, 9), V=rows(kv, 10), **cache, cu=cu, start=start, max_n=most), ["K", "V"]),
            "mp_attn_cache_fwd": (dict(Q=rows(heads, 11), O=rows(heads, 12), LSE=torch.full((heads, total), nan, **f32), **cache,
                                       cu_q=cu, lens=lens, max_q=most,
                                       workspace=torch.zeros(mp.mp_attn_cache_workspace_bytes(heads, kv, d, most),
                                                             dtype=torch.uint8, device="cuda")), ["O", "LSE"]),
        }

    def run(self, name, **change):
        args, out = self.calls[name]
        args = dict(args, **change)
        getattr(mp, name)(**args)
        torch.cuda.synchronize()
        return [args[k].clone().view(torch.uint8) for k in out]


NAMES = ["mp_qk_norm_rope", "mp_qk_norm_rope_bwd", "mp_kv_cache_write", "mp_kv_cache_read", "mp_attn_cache_fwd"]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("strided,T", [(False, 7), (True, 7), (True, 1), (False, 1)])
def test_ordinary_calls_take_the_extension_and_answer_alike(monkeypatch, name, strided, T):
    rec = _Recorder(mp._fast())
    monkeypatch.setattr(mp, "_bind", rec)
    got = Step(strided, T).run(name)
    assert rec.answers == [0]
    monkeypatch.setattr(mp, "_bind", _Off())
    want = Step(strided, T).run(name)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name,change", [
    ("mp_qk_norm_rope", dict(base=10000)), ("mp_qk_norm_rope", dict(sections=[16, 16])),
    ("mp_qk_norm_rope", dict(q_heads=8, wk=None)), ("mp_qk_norm_rope_bwd", dict(q_heads=0, wq=None)),
    ("mp_kv_cache_read", dict(start=None)), ("mp_attn_cache_fwd", dict(scale=1)),
])
def test_calls_out_of_the_ordinary_answer_as_before(monkeypatch, name, change):
    got = Step().run(name, **change)
    monkeypatch.setattr(mp, "_bind", _Off())
    assert all(torch.equal(a, b) for a, b in zip(got, Step().run(name, **change)))


def _wrong(step, name):
    """Each argument of the call once as another type, another shape, on the host, with stretched strides and absent."""
    args, _ = step.calls[name]
    for key, v in args.items():
        if isinstance(v, torch.Tensor):
            yield key, v.to(torch.float64)
            yield key, v.cpu()
            yield key, v.unsqueeze(0)
            if v.dim() > 1 and v.shape[-1] > 1:
                yield key, v.transpose(-1, -2)
            if key != "workspace":
                yield key, torch.cat([v, v])
            yield key, None
            yield key, 5
        elif isinstance(v, int):
            yield key, "x"
            yield key, 1 << 40
            yield key, -1
            yield key, None
        else:
            yield key, ()
            yield key, (16,) * 5
            yield key, (16, "x")
    yield "stream", "x"
    if "cache" in name:
        yield "d_status", torch.zeros(2, dtype=torch.int32, device="cuda")
        yield "d_status", torch.zeros(1, device="cuda")


@pytest.mark.parametrize("name", NAMES)
def test_refusals_are_the_same(monkeypatch, name):
    step = Step()

    def answer(key, value):
        try:
            step.run(name, **{key: value})
        except Exception as e:
            return type(e), str(e)
        return None

    bind = mp._fast()
    refused = 0
    for key, value in _wrong(step, name):
        monkeypatch.setattr(mp, "_bind", bind)
        got = answer(key, value)
        monkeypatch.setattr(mp, "_bind", _Off())
        assert got == answer(key, value), (key, value)
        refused += got is not None
    assert refused > 20


def test_status_word_and_streams():
    step = Step()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = step.run("mp_attn_cache_fwd", d_status=status)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for how in (s, s.cuda_stream):
        assert all(torch.equal(a, b) for a, b in zip(step.run("mp_attn_cache_fwd", d_status=status, stream=how), want))
    assert int(status) == 0
    bad = step.calls["mp_attn_cache_fwd"][0]["page_table"].clone()
    bad[0, 0] = 1 << 20
    step.run("mp_attn_cache_fwd", d_status=status, page_table=bad)
    assert int(status) != 0


def test_threads_call_at_once():
    steps = [Step() for _ in range(4)]
    want = Step().run("mp_attn_cache_fwd")
    got = [None] * len(steps)

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(50):
                got[i] = steps[i].run("mp_attn_cache_fwd")
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(steps))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))
