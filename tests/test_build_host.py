"""The build's decisions about the binding's marshalling module (no GPU)."""
import os
import sys

from sliding_window_attention_gb300 import build


def test_the_library_builds_without_pytorch(monkeypatch, tmp_path):
    """The C ABI needs no PyTorch: without one, the library is built and the marshalling module left out."""
    build.build()
    module = tmp_path / "_marshal.so"
    monkeypatch.setattr(build, "MARSHAL", str(module))
    monkeypatch.setitem(sys.modules, "torch", None)
    assert os.path.exists(build.build()) and not module.exists()
