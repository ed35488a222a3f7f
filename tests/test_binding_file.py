"""The compiled part of the binding: who needs it, and which file it is."""

import importlib.util
import os
import subprocess
import sys
import types

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "paged_kv_cache_sa_b200")


def test_only_the_calls_that_use_it_need_it(tmp_path):
    """A tree with the library alone: everything but append_kv and attend_chunk is there, and those
    two say what is missing."""
    pkg = tmp_path / "paged_kv_cache_sa_b200"
    (pkg / "lib").mkdir(parents=True)
    os.symlink(os.path.join(PKG, "__init__.py"), pkg / "__init__.py")
    os.symlink(os.path.join(PKG, "lib", "libsa.so"), pkg / "lib" / "libsa.so")
    # (the package looks for its files beside the path it was imported from)
    code = """
import torch
import paged_kv_cache_sa_b200 as sa
g = sa.Geometry(B=2, Hq=8, Hkv=2, Dk=128, Dv=128, P=16, max_pages=64, n_pool=256)
assert sa.decode_workspace_size(g, 512) > 0 and sa.chunk_workspace_size(g, 4) > 0
x = torch.zeros(1, 8, 128, dtype=torch.bfloat16)
for call in (lambda: sa.append_kv(g, x, x, x, x, x, x, x, None),
             lambda: sa.attend_chunk(g, x, x, x, x, x, x, 0.1, None)):
    try:
        call()
    except ImportError as e:
        assert "is not built" in str(e), e
    else:
        raise AssertionError("no ImportError")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_another_torch_is_another_file(monkeypatch):
    """The compiled part is linked to one torch and one Python: under another version it is built
    anew, however recent the file of the old one, and the old one is not loaded."""
    spec = importlib.util.spec_from_file_location("_sa_build", os.path.join(PKG, "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    b.build_binding()  # up to date
    made = []

    def compiler(cmd, **kw):
        made.append(cmd[cmd.index("-o") + 1])
        open(made[-1], "w").close()
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")
    with monkeypatch.context() as m:
        m.setattr(b.subprocess, "run", compiler)
        assert os.path.exists(b.build_binding()) and not made
        m.setattr(torch, "__version__", "0.0.other")
        path = b.build_binding()
        try:
            assert len(made) == 1 and os.path.getsize(path) == 0
        finally:
            if made:
                os.remove(path)
    import paged_kv_cache_sa_b200 as sa
    assert os.path.samefile(sa.binding_path(), b.build_binding())
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "0.0.other")
        with pytest.raises(ImportError, match="is not built"):
            sa._load_binding(sa.lib)
