"""The longest-request hint of the attention calls on the GPU."""
import ctypes as C

import pytest
import torch

import sparse_attention_indexer_block_gb300 as saib
from sparse_attention_indexer_block_gb300 import binding
from test_gpu_attend import BF, DEV, Batch, _lib  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hint", [1, 2, 3, 100, 2 ** 31 - 1])
def test_a_hint_past_the_tokens_means_all_tokens(hint):
    """No request has more new tokens than the call: a small step that needs no workspace needs none
    either when the hint is a capacity."""
    b = Batch([1, 1], [1000, 300], 16, 2, 128, BF, seed=600)
    want = b.attend()
    out, lse = torch.empty_like(b.q), torch.empty((2, 16), device=DEV)
    a = binding.Attend(
        q=b.q.data_ptr(), k=b.k.data_ptr(), v=b.v.data_ptr(), block_table=b.table.data_ptr(),
        seq_lens=b.lens.data_ptr(), query_start_loc=b.start.data_ptr(), out=out.data_ptr(), lse=lse.data_ptr(),
        q_stride_token=b.q.stride(0), q_stride_head=b.q.stride(1), k_stride_page=b.k.stride(0),
        k_stride_token=b.k.stride(1), k_stride_head=b.k.stride(2), v_stride_page=b.v.stride(0),
        v_stride_token=b.v.stride(1), v_stride_head=b.v.stride(2), num_pages=b.k.shape[0],
        bt_stride=b.table.stride(0), bt_width=b.width, num_reqs=2, num_tokens=2, num_heads=16, num_kv_heads=2,
        head_dim=128, dtype=0, max_query_len=hint, scale=128 ** -0.5)
    assert saib.load().indexer_attend_paged(C.byref(a), torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    b.check((out, lse), b.reference())
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
