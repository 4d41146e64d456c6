"""Tensors of another GPU than the current one are refused: a kernel would take their addresses for its own."""
import inspect

import pytest
import torch

import tensor_transformer_layer_gb300 as mp
from test_cache_binding import bind  # noqa: F401 (a fixture)

NAMES = ["mp_qk_norm_rope", "mp_qk_norm_rope_bwd", "mp_kv_cache_write", "mp_kv_cache_read", "mp_attn_cache_fwd"]
OTHERS = {"max_n", "max_q", "q_heads", "sections", "base", "eps", "interleaved", "per_axis", "causal", "scale", "stream"}


class Elsewhere(torch.Tensor):
    """Says that it lies on the second GPU."""

    @staticmethod
    def __new__(cls):
        return torch.Tensor._make_wrapper_subclass(cls, (2, 4, 64), dtype=torch.bfloat16, device="cpu", dispatch_device=True)

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        if func is torch.ops.prim.device.default:
            return torch.device("cuda:1")
        raise RuntimeError(f"{func} is not answered")


@pytest.mark.parametrize("name", NAMES)
def test_each_tensor_of_another_device_is_refused(bind, monkeypatch, name):  # noqa: F811
    monkeypatch.setattr(mp, "_current_device", lambda: 0)
    call = getattr(mp, name)
    ints = {k: 1 for k in ("max_n", "max_q", "q_heads")}
    tensors = [k for k in inspect.signature(call).parameters if k not in OTHERS]
    assert len(tensors) >= 5
    for k in tensors:
        args = {t: torch.zeros(2, 4, 64, dtype=torch.bfloat16) for t in tensors}
        args[k] = Elsewhere()
        args.update({n: v for n, v in ints.items() if n in inspect.signature(call).parameters})
        if "sections" in inspect.signature(call).parameters:
            args["sections"] = (32,)
        with pytest.raises(ValueError, match=f"^{k} lies on cuda:1, the current device is cuda:0"):
            call(**args)


@pytest.mark.gpu
def test_the_current_device_is_asked_for():
    x = torch.zeros(3, device="cuda")
    mp._here(x=x, y=None, z=torch.zeros(3))
    assert mp._current_device() == torch.cuda.current_device()
