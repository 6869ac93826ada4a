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


def test_a_module_of_another_pytorch_is_built_again(monkeypatch, tmp_path):
    module = tmp_path / "_marshal.so"
    monkeypatch.setattr(build, "MARSHAL", str(module))
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    assert build._marshal_due("2.9.1")
    module.write_bytes(b"")
    assert build._marshal_due("2.9.1")  # built against an unknown one
    with open(build._marshal_stamp(), "w") as f:
        f.write("2.9.1")
    assert not build._marshal_due("2.9.1") and build._marshal_due("2.11.0") and build._marshal_due("2.9.1", force=True)
    assert not build._marshal_due(None)
    os.utime(module, (0, 0))  # older than its sources
    assert build._marshal_due("2.9.1")
