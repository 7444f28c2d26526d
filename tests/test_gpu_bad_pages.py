"""Pages that lie outside the cache, on the GPU: the keys of one that is needed count as zeros and
are reported, one that a window hides from every token is neither used nor reported."""
import pytest
import torch

import sparse_attention_indexer_block_gb300 as saib
from test_gpu_attend import BF, DEV, FP, PAGE, Batch, _lib  # noqa: F401
from test_gpu_attend_units import _wide

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
