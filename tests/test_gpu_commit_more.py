"""Commits on the GPU: nothing accepted of trees of many nodes."""
import pytest
import torch

import sparse_attention_indexer_block_gb300 as saib
from test_gpu_attend import DEV, _lib  # noqa: F401
from test_gpu_tree import Caches

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
