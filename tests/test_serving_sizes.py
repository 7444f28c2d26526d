"""Workspaces of the attention calls, on the CPU: one that was sized for some sizes holds for every
call of at most those."""
import contextlib
import ctypes as C
import itertools

import pytest
import torch

import sparse_attention_indexer_block_gb300 as saib
from sparse_attention_indexer_block_gb300 import binding
from sparse_attention_indexer_block_gb300 import build as libbuild


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return saib.load()


def _bytes(lib, tokens, reqs, heads, kv, dim):
    n = C.c_size_t(0)
    assert lib.indexer_attend_workspace_bytes(tokens, reqs, heads, kv, dim, C.byref(n)) == 0
    return n.value


@pytest.mark.parametrize("tokens,reqs", [(1, 1), (130, 7), (100000, 1), (8192, 600)])
def test_a_workspace_holds_for_smaller_sizes(lib, tokens, reqs):
    for heads, kv, dim in itertools.product((1, 8, 40, 64), (1, 2, 8, 64), (64, 128)):
        if heads % kv:
            continue
        most = _bytes(lib, tokens, reqs, heads, kv, dim)
        for t, r, h, k, d in itertools.product((1, tokens // 2 + 1, tokens), (1, reqs // 2 + 1, reqs),
                                               (1, 5, 8, 40, 64), (1, 2, 5, 8, 40, 64), (64, 128)):
            if h <= heads and k <= kv and d <= dim and h % k == 0:
                assert _bytes(lib, t, r, h, k, d) <= most, (heads, kv, dim, t, r, h, k, d)


def test_a_workspace_is_sized_for_its_own_device(monkeypatch):
    now, asked = [0], []

    @contextlib.contextmanager
    def device(d):
        keep, now[0] = now[0], torch.device(d).index
        yield
        now[0] = keep

    class Lib:
        @staticmethod
        def indexer_attend_workspace_bytes(*args):
            asked.append(now[0])
            args[-1]._obj.value = 4096
            return 0

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch, "empty", lambda n, dtype, device: (n, torch.device(device)))
    monkeypatch.setattr(binding, "load", Lib)
    binding._attend_workspace_bytes.cache_clear()
    try:
        assert saib.attend_workspace(7, 2, 8, 2, 128, "cuda:3") == (4096, torch.device("cuda:3"))
        assert asked == [3] and now == [0]
        assert saib.attend_workspace(7, 2, 8, 2, 128, "cuda:1")[0] == 4096 and asked == [3, 1]
    finally:
        binding._attend_workspace_bytes.cache_clear()
