"""The drafted trees of examples/paged_serving.py: the outputs against the formula in 64 bits on the keys
that each node sees, and the caches' state after the kept paths."""
import torch
import pytest

from test_gpu_attend import DEV, _lib  # noqa: F401
from test_gpu_serving_example import _attention, example  # noqa: F401

pytestmark = pytest.mark.gpu


def test_drafted_trees(example):  # noqa: F811
    m = example
    r = m.run_drafts(DEV)
    torch.cuda.synchronize()
    pool = r["pool"]
    assert int(pool.err) == 0
    # (as in the serving loop's test: weights, outputs and the products of entries rounded to bf16)
    v_size = max((h @ pool.wv).abs().max().item() for h in r["history"])
    for history, x, dense, sparse in r["steps"]:
        v_step = max(v_size, (x @ pool.wv).abs().max().item())
        at = 0
        for h, tree in zip(history, r["trees"]):
            chains = []
            for i, p in enumerate(tree):
                chains.append((chains[p] if p >= 0 else []) + [at + i])
                want = _attention(m, pool, torch.cat([h, x[chains[i]]]), x[at + i])
                assert (dense[at + i].double() - want).abs().max() <= 3 * 2.0 ** -8 * v_step
                if h.shape[0] <= m.TOPK:      # every key before the tree is selected
                    assert (sparse[at + i].double() - want).abs().max() <= 3 * 2.0 ** -8 * v_step
            at += len(tree)
        assert torch.isfinite(sparse).all()
    assert pool.lens.tolist() == [h.shape[0] for h in r["history"]]
    held = sum(-(-h.shape[0] // m.PAGE) for h in r["history"])
    assert int(pool.refs.sum()) == held
    for row, h in enumerate(r["history"]):
        pos = torch.arange(h.shape[0], device=DEV)
        page, slot = pool.table[row, pos // m.PAGE].long(), pos % m.PAGE
        for cache, w in ((pool.k, pool.wk), (pool.v, pool.wv)):
            want = (h @ w).view(-1, m.KV_HEADS, m.DIM)
            # (16-bit products of a batch and of a single row may differ in their last place)
            assert ((cache[page, slot] - want).abs() <= 2.0 ** -8 * (want.abs() + v_size)).all()
