"""examples/paged_serving.py on the GPU: its outputs against the formula in 64
bits on the tokens each request has seen, and the pool's state."""
import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def example():
    from sparse_attention_indexer_block_gb300 import build as libbuild
    libbuild.build()
    torch.cuda.set_device(DEV)
    spec = importlib.util.spec_from_file_location("paged_serving",
                                                  os.path.join(ROOT, "examples", "paged_serving.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _attention(m, pool, seen, x, window=0, sinks=0):
    """Of token x (the last of seen) in 64 bits, on the 16-bit entries the caches hold."""
    q = (x[None] @ pool.wq).view(m.HEADS, m.DIM).double()
    k = (seen @ pool.wk).view(-1, m.KV_HEADS, m.DIM).double()
    v = (seen @ pool.wv).view(-1, m.KV_HEADS, m.DIM).double()
    n, g = seen.shape[0], m.HEADS // m.KV_HEADS
    see = torch.ones(n, dtype=torch.bool, device=DEV)
    if window:
        pos = torch.arange(n, device=DEV)
        see = (n - 1 - pos < window) | (pos < sinks)
    s = torch.einsum("hd,nhd->hn", q, k.repeat_interleave(g, 1)) / math.sqrt(m.DIM)
    p = torch.softmax(s.masked_fill(~see, -math.inf), -1)
    return torch.einsum("hn,nhd->hd", p, v.repeat_interleave(g, 1))


def test_serving_loop(example):
    m = example
    r = m.run(DEV)
    torch.cuda.synchronize()
    pool = r["pool"]
    assert int(pool.err) == 0
    a, b = r["tokens"]
    # The library's outputs round weights and outputs to bf16 (2^-8 of the values' weighted mean
    # size, about 0.8 of the largest |v| here at most, each); the 16-bit products of the caches'
    # entries may differ in their last place between a batch and a single row (2^-8 of |v|).
    def close(got, want, v_size):
        assert (got.double() - want).abs().max() <= 3 * 2.0 ** -8 * v_size

    v_size = (a @ pool.wv).abs().max().item()
    first, second = r["prompt"][0][0], r["prompt"][1][0]
    for i in (0, 63, 64, 999):
        close(first[i], _attention(m, pool, a[:i + 1], a[i]), v_size)
    close(second[-1], _attention(m, pool, a, a[-1]), v_size)
    close(r["prompt"][0][1][-1], _attention(m, pool, b, b[-1]), v_size)
    # forks that take the same token as their parents give the same outputs, bit for bit
    sparse, windowed = r["decoded"][0]
    for child, parent in ((2, 0), (3, 1), (4, 1)):
        assert torch.equal(windowed[child], windowed[parent])
    history = [torch.cat([h] + [x[i:i + 1] for x in r["steps"]]) for i, h in enumerate((a, b, a, b, b))]
    sparse, windowed = r["decoded"][-1]
    for i, h in enumerate(history):
        close(windowed[i], _attention(m, pool, h, h[-1], m.WINDOW, m.SINKS), v_size)
        if h.shape[0] <= m.TOPK:      # every key is selected
            close(sparse[i], _attention(m, pool, h, h[-1]), v_size)
    # pages: 24 of the first prompt and 6 of the second, 4 + 1 last ones of the forks and of growth
    assert r["live"] < r["used"]
    live = r["live"]
    held = torch.unique(torch.cat([pool.table[i, :-(-int(pool.lens[i]) // m.PAGE)] for i in (1, 2, 4)]))
    assert pool.lens.tolist() == [0, 339, 1506, 0, 339, 0, 0, 0]
    assert int(pool.refs.sum()) == sum(-(-int(n) // m.PAGE) for n in pool.lens)
    assert held.numel() == int((pool.refs > 0).sum()) and held.max() < live + 3
    for out in r["more"]:
        assert all(torch.isfinite(o).all() for o in out)
