"""The prefill selection handed to attention as it is: indexer_prefill_topk's lists into
indexer_attend_selected over one block table, against the formula in 64 bits on those lists
(tolerances as in test_gpu_attend)."""
import pytest
import torch

import synth
import sparse_attention_indexer_block_gb300 as saib
from test_gpu_attend import BF, DEV, FP, PAGE, Batch, _lib  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ql,kl,topk,heads,kv,dtype,dim", [([200, 64, 1], [900, 64, 300], 128, 16, 2, BF, 128),
                                                           ([300, 7], [300, 1500], 512, 32, 8, FP, 64)])
def test_prefill_lists(ql, kl, topk, heads, kv, dtype, dim):
    p = synth.make_prefill(seed=55, seq_lens=kl, query_lens=ql)
    b = Batch(ql, kl, heads, kv, dim, dtype, seed=700)
    index = torch.zeros((b.k.shape[0], synth.PAGE_BYTES), dtype=torch.uint8, device=DEV)
    for r, n in enumerate(kl):
        pages = -(-n // PAGE)
        index[b.table[r, :pages].long()] = p.cache.to(DEV)[p.block_table[r, :pages].long().to(DEV)]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    idx = saib.indexer_prefill_topk(p.q.to(DEV), p.w.to(DEV), index, b.table, b.lens, b.start, p.seq_lens,
                                    p.query_lens, topk, dev_error=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    # a row's list is of its own causal keys, as many as there are or topk
    row = 0
    for q, n in zip(ql, kl):
        for seen in range(n - q + 1, n + 1):
            got = idx[row][idx[row] >= 0]
            assert got.numel() == min(topk, seen) == torch.unique(got).numel() and int(got.max()) < seen
            row += 1
    b.check(b.attend_selected(idx), b.reference(indices=idx))
