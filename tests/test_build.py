"""The build and the loading of the library and its marshalling module, on the CPU."""
import os
import shutil
import subprocess
import sys

import pytest
import torch

from sparse_attention_indexer_block_gb300 import build as libbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    return libbuild.build()


def test_a_build_is_stale_for_another_torch_or_recipe(lib, monkeypatch):
    assert not libbuild._stale()
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "0.0.1")
        assert libbuild._stale()
    real, recipe = os.path.getmtime, os.path.abspath(libbuild.__file__)
    with monkeypatch.context() as m:
        m.setattr(os.path, "getmtime", lambda p: real(lib) + 10 if os.path.abspath(p) == recipe else real(p))
        assert libbuild._stale()
    assert not libbuild._stale()


def _run(code, *args):
    r = subprocess.run([sys.executable, "-c", code, *args], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr


def test_every_call_uses_the_library_that_was_loaded(lib, tmp_path):
    other = tmp_path / "libother.so"
    shutil.copy(lib, other)
    _run("""
import sys
import sparse_attention_indexer_block_gb300 as saib
from sparse_attention_indexer_block_gb300 import binding
saib.load(sys.argv[1])
assert saib.indexer_status_string(0) == "ok"
try:
    saib.indexer_attend_paged(*[None] * 6)
    raise SystemExit("not refused")
except saib.IndexerError:
    pass
maps = open("/proc/self/maps").read()
assert sys.argv[1] in maps and "libsaib.so" not in maps
""", str(other))


def test_calls_that_pass_by_the_module_do_without_it(lib):
    _run("""
import sys
sys.modules["sparse_attention_indexer_block_gb300._marshal"] = None
import sparse_attention_indexer_block_gb300 as saib
saib.load()
assert saib.indexer_status_string(0) == "ok"
try:
    saib.indexer_attend_paged(*[None] * 6)
    raise SystemExit("no error")
except RuntimeError as e:
    assert "not built" in str(e)
""")


def test_a_library_that_lacks_a_function_is_refused(lib):
    import ctypes

    from sparse_attention_indexer_block_gb300 import binding
    with pytest.raises(RuntimeError, match="indexer_attend_paged"):
        binding._native().bind(ctypes.CDLL(None)._handle)


def test_a_build_without_the_module_leaves_the_library(lib, tmp_path, monkeypatch):
    for name in ("LIB", "MARSHAL", "OBJECTS"):
        monkeypatch.setattr(libbuild, name, str(tmp_path / name))
    monkeypatch.setattr(libbuild, "SOURCES", ["no_alloc.cu"])
    monkeypatch.setattr(libbuild, "_marshal_command", lambda nvcc, obj: ["false"])
    monkeypatch.setattr(subprocess, "run", lambda cmd, **kw: open(cmd[cmd.index("-o") + 1], "w").close())
    with pytest.raises(RuntimeError, match="marshal.cpp"):
        libbuild.build(force=True)
    assert (tmp_path / "LIB").exists() and not (tmp_path / "MARSHAL").exists()
