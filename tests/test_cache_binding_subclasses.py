"""Tensors that answer like no ordinary one: the extension leaves them to the checks in Python, without an error left behind."""
import ctypes

import pytest
import torch

from test_cache_binding import COUNTS, bind  # noqa: F401 (a fixture)


class Raising(torch.Tensor):
    """Asks Python where it lies and how large it is; the questions from `silent` on raise."""

    @staticmethod
    def __new__(cls, shape, dtype, silent):
        t = torch.Tensor._make_wrapper_subclass(cls, shape, dtype=dtype, device="cpu", dispatch_device=True,
                                                dispatch_sizes_strides_policy="sizes")
        t.silent = silent
        return t

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        if func is torch.ops.prim.device.default and not args[0].silent:
            return torch.device("cuda:0")
        raise RuntimeError(f"{func} is not answered")


def _left_alone(f, args):
    answer = f(*args)
    ctypes.pythonapi.PyErr_Occurred()  # raises an error that is still set
    assert answer is None


# arguments before which the extension looks at nothing else, and their type
FIRST = {"qk_norm_rope": (0, torch.bfloat16, {5: 3, 6: (32,), 9: 0}),
         "qk_norm_rope_bwd": (0, torch.bfloat16, {9: 3, 10: (32,), 13: 0}),
         "kv_cache_write": (2, torch.float8_e4m3fn, {}), "kv_cache_read": (2, torch.float8_e4m3fn, {}),
         "attn_cache_fwd": (1, torch.float8_e4m3fn, {})}


@pytest.mark.parametrize("name", FIRST)
@pytest.mark.parametrize("silent", [True, False])
def test_a_tensor_that_raises_is_left_to_the_checks(bind, name, silent):  # noqa: F811
    at, dtype, others = FIRST[name]
    args = [None] * COUNTS[name]
    for i, v in others.items():
        args[i] = v
    args[at] = Raising((2, 4, 64) if dtype is torch.bfloat16 else (2, 2, 16, 64), dtype, silent)
    _left_alone(getattr(bind, name), args)


def test_the_checks_answer_for_it(bind):  # noqa: F811
    import tensor_transformer_layer_gb300 as mp
    x = Raising((2, 4, 64), torch.bfloat16, True)
    with pytest.raises(RuntimeError, match="not answered") as e:
        mp.mp_qk_norm_rope(x, x, None, None, None, q_heads=4, sections=(32,))
    assert e.value.__cause__ is None
