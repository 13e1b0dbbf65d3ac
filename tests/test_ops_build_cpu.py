"""The build's steps on a host without torch."""
import os
import sys

from fp32_gemm_f32_amd import build


def test_the_library_is_usable_without_torch(monkeypatch, capsys):
    """No torch: the extension for its tensors is left out, with a word, and nothing fails."""
    monkeypatch.setitem(sys.modules, "torch", None)      # an import of it now raises ImportError
    out = os.path.join(build.PKG, "_torch_calls.so")
    before = os.stat(out).st_mtime_ns if os.path.exists(out) else None
    assert build.build_calls() is None
    assert "torch" in capsys.readouterr().err
    assert before == (os.stat(out).st_mtime_ns if os.path.exists(out) else None)
