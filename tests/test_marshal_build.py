"""The marshalling module is the running Python's and PyTorch's, and the C library does not depend on it."""
import pytest

from routed_moe_expert_gb300 import _build
from routed_moe_expert_gb300 import binding as B


@pytest.mark.parametrize("was", ["Python 3.1, PyTorch 1.0", None])
def test_a_module_of_another_pytorch_is_rebuilt_and_not_loaded(built_lib, monkeypatch, tmp_path, was):
    abi = tmp_path / "abi"
    if was:
        abi.write_text(was)
    monkeypatch.setattr(_build, "MARSHAL_ABI", str(abi))
    monkeypatch.setattr(B, "_marshal", None)
    with pytest.raises(B.MoELoRAError, match="built against"):
        B._native()
    rebuilt = []
    monkeypatch.setattr(_build, "_build_marshal", lambda verbose: (rebuilt.append(1), abi.write_text(_build.marshal_abi())))
    monkeypatch.setattr(_build, "_build_library", lambda verbose: pytest.fail("the library is up to date"))
    _build.build()
    _build.build()
    assert rebuilt == [1]
    assert B._native() is not None


def test_the_library_is_built_when_the_module_cannot_be(monkeypatch, tmp_path):
    def fails(verbose):
        raise RuntimeError("g++ failed")
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(_build, "BUILD", str(tmp_path))
    monkeypatch.setattr(_build, "SOURCES", ["linear.cu"])      # (one file stands for the library)
    monkeypatch.setattr(_build, "_build_marshal", fails)
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        _build.build(force=True)
    assert (tmp_path / "lib.so").exists()
