"""The build and the loading of the library and its marshalling module, on the CPU."""
import os

import pytest
import torch

from sparse_attention_indexer_block_gb300 import build as libbuild

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
