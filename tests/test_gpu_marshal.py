"""What the native marshalling of the calls does beside their work: errors of torch stay torch's own."""
import pytest
import torch

import sparse_attention_indexer_block_gb300 as saib
from test_gpu_attend import BF, DEV, Batch, _lib  # noqa: F401
from test_gpu_tree import TreeBatch, _i32

pytestmark = pytest.mark.gpu


@pytest.fixture
def little_memory():
    """An allocator that hands out a hundredth of the device (no memory is taken)."""
    torch.cuda.empty_cache()
    torch.cuda.set_per_process_memory_fraction(0.01)
    yield
    torch.cuda.set_per_process_memory_fraction(1.0)


def test_outputs_that_do_not_fit_are_out_of_memory(little_memory):
    tokens = 1 << 24
    b, t = Batch([1], [100], 4, 2, 128, BF), TreeBatch([1], [100], 4, 2, 128, BF)
    want, tree = b.attend(), t.attend_tree()
    q, start = b.q.expand(tokens, 4, 128), _i32([0, tokens])
    flat = torch.zeros(1, dtype=torch.int32, device=DEV)
    calls = [lambda: saib.indexer_attend_paged(q, b.k, b.v, b.table, b.lens, start),
             lambda: saib.indexer_attend_selected(q, b.k, b.v, b.table, torch.zeros((1, 1), dtype=torch.int32, device=DEV).expand(tokens, 1), start),
             lambda: saib.indexer_attend_tree(q, b.k, b.v, b.table, b.lens, start, torch.zeros((tokens, 1), dtype=torch.int32, device=DEV)),
             lambda: saib.indexer_plan_tree(torch.zeros(tokens, dtype=torch.int32, device=DEV), b.lens, start, 64 * 64),
             lambda: saib.indexer_append_kv(b.q[:, :2].expand(tokens, 2, 128), b.q[:, :2].expand(tokens, 2, 128), b.k, b.v,
                                            torch.full((tokens,), -1, dtype=torch.int64, device=DEV), q=q,
                                            positions=flat.expand(tokens).contiguous(),
                                            rotary=torch.ones((1, 128), device=DEV))]
    for call in calls:
        with pytest.raises(torch.OutOfMemoryError):
            call()
    # and the next calls are as before
    assert all(torch.equal(a, c) for a, c in zip(b.attend(), want))
    assert all(torch.equal(a, c) for a, c in zip(t.attend_tree(), tree))
