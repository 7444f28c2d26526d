"""Commits on the GPU: nothing accepted of trees of many nodes; the caches of many layers, which take several launches."""
import pytest
import torch

import sparse_attention_indexer_block_gb300 as saib
from test_gpu_attend import DEV, PAGE, _lib  # noqa: F401
from test_gpu_tree import Caches, _i32, _paths

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pools", [0, 2, 4])
@pytest.mark.parametrize("ql,kl", [([2100, 0, 5, 3000], [2200, 10, 5, 3001]), ([64] * 50, [64 + 9 * i for i in range(50)])])
def test_commit_of_lists_without_columns(ql, kl, pools):
    """The length is written when every thread has read it, without lists to go through too."""
    c = Caches(ql, kl, seed=12)
    want = c.expected([[]] * len(ql))
    saib.indexer_commit_tree(c.pools[:pools], c.table, c.lens, c.start,
                             torch.empty((len(ql), 0), dtype=torch.int32, device=DEV), ref_counts=c.refs, dev_error=c.err)
    torch.cuda.synchronize()
    assert int(c.err) == 0
    c.check(want)


class Layers:
    """The caches of n layers, small and wide tokens in turn, whose pools make `entries` entries of a launch's 48 (an fp8
    index cache is two)."""

    def __init__(self, c, entries, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        n, self.c, self.pools, at, layer = c.index.shape[0], c, [], 0, 0
        while at < entries:
            kv, dim = [(1, 64), (8, 128), (3, 64)][layer % 3]
            for kind in ("index", "k", "v", "mx"):
                size = 2 if kind == "index" else 1
                if at + size > entries or (kind == "mx" and layer % 2):
                    continue
                if kind in "kv":
                    shape = (n, kv, PAGE, dim) if layer % 4 == 1 else (n, PAGE, kv, dim)
                    t = torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)
                    self.pools.append(t.transpose(1, 2) if layer % 4 == 1 else t)
                else:
                    self.pools.append(torch.randint(0, 256, (n, 8448 if kind == "index" else 4352), generator=g,
                                                    device=DEV, dtype=torch.uint8))
                at += size
            layer += 1
        assert len(saib.binding._native().token_pools(self.pools)) == entries

    def tokens(self):
        """Every pool as [pages, 64, bytes or values]."""
        out = []
        for t in self.pools:
            n = t.shape[0]
            if t.dtype == torch.uint8 and t.shape[1] == 8448:
                out += [t[:, :8192].reshape(n, PAGE, 128).clone(), t[:, 8192:].reshape(n, PAGE, 4).clone()]
            else:
                out.append(t.reshape(n, PAGE, -1).clone())
        return out

    def expected(self, paths):
        self.c.tokens = self.tokens      # (Caches.expected moves what tokens() gives)
        return self.c.expected(paths)

    def check(self, want):
        caches, refs, lens = want
        for i, (got, c) in enumerate(zip(self.tokens(), caches)):
            assert torch.equal(got, c), f"entry {i}"
        assert self.c.refs.tolist() == refs and self.c.lens.tolist() == lens


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("entries", [47, 48, 49, 96, 97, 100, 145])
def test_commit_of_many_pools(entries, graph):
    """Lengths and references follow with the last launch only, and each has its own clusters."""
    ql, kl = [20, 0, 64, 3, 70], [200, 7, 64, 130, 129]
    c = Caches(ql, kl, seed=entries)
    layers = Layers(c, entries, seed=entries)
    paths = _paths(ql, 5, most=40)
    want = layers.expected(paths)
    most = max(len(p) for p in paths)
    accepted = _i32([list(p) + [-1] * (most - len(p)) for p in paths])

    def call():
        saib.indexer_commit_tree(layers.pools, c.table, c.lens, c.start, accepted, ref_counts=c.refs, dev_error=c.err)

    if graph:
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            call()
        captured.replay()
    else:
        call()
    torch.cuda.synchronize()
    assert int(c.err) == 0
    layers.check(want)
