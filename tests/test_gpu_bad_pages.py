"""Pages that lie outside the cache, on the GPU: one that a window hides from every token is neither
used nor reported."""
import pytest
import torch

import sparse_attention_indexer_block_gb300 as saib
from test_gpu_attend import BF, DEV, FP, PAGE, Batch, _lib  # noqa: F401
from test_gpu_attend_units import _wide

pytestmark = pytest.mark.gpu


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
