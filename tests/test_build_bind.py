"""The short way from torch into the library is built where it can be; the library does not depend on it."""

import os
import shutil

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytest.importorskip("torch")


@pytest.mark.parametrize("fault", ["source", "compiler"])
def test_a_failing_compiler_leaves_the_library_alone(fault, tmp_path, monkeypatch, capsys):
    if not os.path.exists(os.path.join(ROOT, "block_scaled_precision_e4m3_amd", "libmxgemm.so")):
        import __graft_entry__
        __graft_entry__.build()
    from block_scaled_precision_e4m3_amd import _build
    bind = tmp_path / "_bind.so"
    bind.write_bytes(b"of an earlier build")
    monkeypatch.setattr(_build, "BIND", str(bind))
    which = shutil.which
    if fault == "source":
        bad = tmp_path / "bind.cpp"
        bad.write_text("#error no such header\n")
        monkeypatch.setattr(_build, "BIND_SOURCE", str(bad))
    else:
        monkeypatch.setattr(_build.shutil, "which", lambda name: str(tmp_path / "none") if name == "g++" else which(name))
    assert _build.build_bind() is None
    assert not os.path.exists(bind), "a binding of an earlier build stayed beside the new library"
    assert "g++ failed" in capsys.readouterr().err
