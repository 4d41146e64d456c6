"""The extension that marshals a decoding step's calls is bound to the torch that it was built for; the library is not."""
import os

import pytest

import tensor_transformer_layer_gb300 as mp
from tensor_transformer_layer_gb300 import build


@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    """A build of one source into a folder of its own."""
    monkeypatch.setattr(build, "LIB_DIR", str(tmp_path))
    monkeypatch.setattr(build, "LIB_PATH", str(tmp_path / "libmptp.so"))
    monkeypatch.setattr(build, "BIND_PATH", str(tmp_path / "_mptp_bind.so"))
    monkeypatch.setattr(build, "BIND_FOR_PATH", str(tmp_path / "_mptp_bind.for"))
    monkeypatch.setattr(build, "sources", lambda: [os.path.join(build.CSRC, "mptp_common.cu")])
    calls = []

    def command(target, obj):
        calls.append(obj)
        return ["cp", build.BIND_SRC, target[:-3] + ".o" if obj else target + ".tmp"]

    monkeypatch.setattr(build, "bind_command", command)
    return calls


def test_built_again_for_another_torch(monkeypatch, elsewhere):
    build.build()
    build.build()
    assert elsewhere == [True, False]  # compiled and linked once
    assert build.bind_built_for() == build.bind_for()
    was = build.bind_for()
    monkeypatch.setattr(build, "bind_for", lambda: was + " patched")
    build.build()
    assert elsewhere == [True, False] * 2 and build.bind_built_for() == was + " patched"
    os.remove(build.BIND_FOR_PATH)  # one of an earlier build, which does not say
    build.build()
    assert elsewhere == [True, False] * 3


def test_library_is_linked_where_the_extension_does_not_compile(monkeypatch, elsewhere):
    monkeypatch.setattr(build, "bind_command", lambda target, obj: ["false"])
    with pytest.raises(RuntimeError, match="extension"):
        build.build()
    assert os.path.exists(build.LIB_PATH) and build.bind_built_for() is None


def test_not_loaded_under_another_torch(monkeypatch):
    build.build()
    monkeypatch.setattr(mp, "_bind", None)
    monkeypatch.setattr(build, "bind_for", lambda: "cpython-312, torch 0.0")
    with pytest.raises(OSError, match="built for .*installed is cpython-312, torch 0.0"):
        mp._fast()
    monkeypatch.undo()
    assert mp._fast()
