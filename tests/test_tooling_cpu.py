"""What the bench and the build say about the sources they were made with."""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)


def test_profiled_traffic_is_of_the_present_forward_kernel():
    import bench
    for name, rec in bench.PROFILED_TRAFFIC.items():
        assert bench.kernel_traffic(name) == rec["bytes"]


def test_library_builds_without_what_the_python_entry_needs(monkeypatch, tmp_path):
    """No torch headers or no g++: the library is there all the same, and the
    Python entry's calls say what is missing."""
    import subprocess

    import pytest

    from sparse_sliding_window_b200 import build as b
    from sparse_sliding_window_b200 import lf_attn as L
    b.build()
    monkeypatch.setattr(b, "BIND", str(tmp_path / "_lf_bind.so"))

    def no_compiler(cmd, *a, **k):
        raise FileNotFoundError(cmd[0])

    monkeypatch.setattr(subprocess, "check_call", no_compiler)
    with pytest.warns(UserWarning, match="_lf_bind"):
        assert b.build() == b.LIB
    with pytest.raises(FileNotFoundError):
        b.build_bind()
    monkeypatch.setattr(L, "_bind", None)
    monkeypatch.setattr(L, "BIND_PATH", b.BIND)
    with pytest.raises(RuntimeError, match="not built"):
        L.lf_rope_fwd(L.make_rope_params(), [], [])


def test_python_entry_is_rebuilt_for_another_torch(monkeypatch, tmp_path):
    import shutil
    import subprocess

    import torch

    from sparse_sliding_window_b200 import build as b
    b.build()
    copy = str(tmp_path / "_lf_bind.so")
    shutil.copy(b.BIND, copy)
    monkeypatch.setattr(b, "BIND", copy)
    calls = []

    def compiler(cmd, *a, **k):
        calls.append(cmd)
        shutil.copy(copy, cmd[cmd.index("-o") + 1])

    monkeypatch.setattr(subprocess, "check_call", compiler)
    assert b.build_bind() == copy and not calls          # up to date
    monkeypatch.setattr(torch, "__version__", "9.9.9+other")
    b.build_bind()
    assert len(calls) == 1
