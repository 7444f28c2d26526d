"""Pages that lie outside the cache, on the GPU: the keys of one that is needed count as zeros and
are reported, one that a window hides from every token is neither used nor reported, and a fork
whose parent's partial last page is one keeps the full pages only."""
import numpy as np
import pytest
import torch

import sparse_attention_indexer_block_gb300 as saib
from test_gpu_attend import BF, DEV, FP, PAGE, Batch, _lib  # noqa: F401
from test_gpu_attend_units import _wide
from test_gpu_pages import Pool, _i32

pytestmark = pytest.mark.gpu

BAD_BLOCK = 1


def _call(b, table, **kw):
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = saib.indexer_attend_paged(b.q, b.k, b.v, table, b.lens, b.start, max(b.ql), dev_error=err, **kw)
    torch.cuda.synchronize()
    return out, lse, int(err.item())


def _hidden(first, column, window, sinks):
    """Whether no token sees a key of the page: its last key has left the window of the first token
    (at position first), its first key is no sink."""
    return window > 0 and column * PAGE + PAGE - 1 <= first - window and column * PAGE >= sinks


# new tokens, keys, whether the table is so wide that units are cut by a plan
BATCHES = [([1, 2], [900, 1000], False), ([1, 2], [900, 1000], True), ([70, 90], [900, 1000], False),
           ([300, 200], [5000, 1000], False), ([1] * 30 + [400], [900] * 30 + [3000], False)]


@pytest.mark.parametrize("window,sinks", [(0, 0), (600, 10)])
@pytest.mark.parametrize("dtype,dim", [(BF, 128), (FP, 64)])
@pytest.mark.parametrize("batch", range(len(BATCHES)))
def test_keys_of_a_page_outside_the_cache_are_zeros(batch, dtype, dim, window, sinks):
    ql, kl, wide = BATCHES[batch]
    b = Batch(ql, kl, 8, 2, dim, dtype, seed=400 + batch)
    if wide:
        _wide(b)
    page = int((set(range(b.k.shape[0])) - set(b.table.flatten().tolist())).pop())
    b.k[page], b.v[page] = 0, 0
    last = len(kl) - 1
    for column in (0, 8, 9, (kl[last] - 1) // PAGE):
        keep = b.table[last, column].item()
        b.table[last, column] = page
        want = b.reference(window=window, sinks=sinks)
        b.table[last, column] = keep
        for bad in (-1, b.k.shape[0], 2 ** 31 - 1, -2 ** 31):
            table = b.table.clone()
            table[last, column] = bad
            first = None
            for _ in range(2):
                out, lse, err = _call(b, table, window=window, sinks=sinks)
                assert err == (0 if _hidden(kl[last] - ql[last], column, window, sinks) else BAD_BLOCK)
                b.check((out, lse), want)
                assert first is None or torch.equal(out, first)
                first = out


@pytest.mark.parametrize("window,sinks", [(1, 0), (70, 0), (70, 5), (129, 70), (64, 64)])
@pytest.mark.parametrize("dtype,dim", [(BF, 128), (FP, 64)])
@pytest.mark.parametrize("batch", range(len(BATCHES)))
def test_pages_hidden_by_a_window_may_be_gone(batch, dtype, dim, window, sinks):
    ql, kl, wide = BATCHES[batch]
    b = Batch(ql, kl, 8, 2, dim, dtype, seed=420 + batch)
    if wide:
        _wide(b)
    out, lse, err = _call(b, b.table, window=window, sinks=sinks)
    assert err == 0
    b.check((out, lse), b.reference(window=window, sinks=sinks))
    for gone in (-1, b.k.shape[0]):
        table, hidden = b.table.clone(), 0
        for r, (q, n) in enumerate(zip(ql, kl)):
            for c in range(-(-n // PAGE)):
                if _hidden(n - q, c, window, sinks):
                    table[r, c] = gone
                    hidden += 1
        assert hidden
        got, glse, err = _call(b, table, window=window, sinks=sinks)
        assert err == 0
        assert torch.equal(got, out) and torch.equal(glse, lse)


@pytest.mark.parametrize("pools", [3, 0])
@pytest.mark.parametrize("bad", [-1, -2 ** 31, "pages", 2 ** 31 - 1])
def test_fork_from_a_bad_last_page(bad, pools):
    p = Pool([100, 200, 64, 7], 2, seed=21, rows=9, pools=pools)
    bad = p.pages if bad == "pages" else bad
    p.table[1, 3] = bad                    # 200 keys: three full pages and a part
    p.up()
    # rows 0 and 3 take the two free pages, though the bad one comes between them
    src, dst, want, short = p.fork([0, 3], [4, 6])
    assert not short
    p.table[5, :3] = p.table[1, :3]        # by hand: the full pages only
    np.add.at(p.refs, p.table[1, :3], 1)
    p.lens[5] = 3 * PAGE
    got = saib.indexer_fork_pages(p.pools, p.t, p.l, p.r, _i32([0, 1, 3]), _i32([4, 5, 6]), dev_error=p.err)
    assert p.error() == BAD_BLOCK
    p.same()
    assert got[0].tolist() == src + [-1] and got[1].tolist() == dst + [-1]
    for a, w in zip(p.pools, want):
        assert torch.equal(a, w)


def test_fork_from_bad_last_pages_when_pages_run_out():
    p = Pool([100, 200, 7], 1, seed=22, rows=8, pools=1)
    p.table[1, 3] = -5
    p.up()
    src, dst, want, short = p.fork([0, 2], [3, 6])     # one free page for two
    assert short
    p.table[4, :3] = p.table[1, :3]
    np.add.at(p.refs, p.table[1, :3], 1)
    p.lens[4] = 3 * PAGE
    got = saib.indexer_fork_pages(p.pools, p.t, p.l, p.r, _i32([0, 1, 2]), _i32([3, 4, 6]), dev_error=p.err)
    assert p.error() == BAD_BLOCK | 64
    p.same()
    assert got[0].tolist() == src + [-1] and got[1].tolist() == dst + [-1]
    assert torch.equal(p.pools[0], want[0])
