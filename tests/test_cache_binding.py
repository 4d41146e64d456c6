"""The extension that marshals a decoding step's calls, without a GPU: it leaves everything that it does not know to the checks."""
import pytest
import torch


@pytest.fixture(scope="module")
def bind():
    from tensor_transformer_layer_gb300 import build
    build.build()
    import tensor_transformer_layer_gb300 as mp
    return mp._fast()


COUNTS = {"qk_norm_rope": 11, "qk_norm_rope_bwd": 15, "kv_cache_write": 12, "kv_cache_read": 12, "attn_cache_fwd": 16}


@pytest.mark.parametrize("name,n", COUNTS.items())
def test_leaves_the_rest_to_the_checks(bind, name, n):
    f = getattr(bind, name)
    for v in (None, 5, 1 << 80, "x", 0.5, (), (1, 2), (1,) * 9, object(), torch.zeros(2, 4, 64, dtype=torch.bfloat16),
              torch.zeros(2, 2, 16, 64, dtype=torch.float8_e4m3fn), torch.zeros(3, dtype=torch.int32), torch.zeros(0),
              torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="meta"), torch.eye(3).to_sparse()):
        assert f(*[v] * n) is None
    with pytest.raises(TypeError):
        f(*[None] * (n - 1))
    with pytest.raises(TypeError):
        f()


def test_missing_extension_is_an_error(monkeypatch):
    import tensor_transformer_layer_gb300 as mp
    monkeypatch.setattr(mp, "_bind", None)
    monkeypatch.setattr(mp, "BIND_PATH", mp.BIND_PATH + ".none")
    with pytest.raises(OSError, match="not built"):
        mp._fast()
