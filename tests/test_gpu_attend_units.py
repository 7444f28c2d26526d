"""Attention of few short units on the GPU: units shared by clusters of one to eight blocks, against
the formula in 64 bits (tolerances as in test_gpu_attend), and next to the same calls with a block
table so wide that their tiles are cut by a plan instead."""
import pytest
import torch

import sparse_attention_indexer_block_gb300 as saib
from test_gpu_attend import BF, DEV, FP, Batch, _lists, _lib  # noqa: F401

pytestmark = pytest.mark.gpu


def _wide(b, width=20000):
    """The batch with a table of that many columns, unused ones invalid."""
    table = torch.full((len(b.kl), width), -7, dtype=torch.int32, device=DEV)
    table[:, :b.width] = b.table
    b.table, b.width = table, width
    return b


# new tokens, keys, heads, kv heads: clusters of 8, 8, 4, 2 and 1 blocks, and too many units for any
UNITS = [
    ([1], [1], 1, 1),
    ([1, 3], [1000, 517], 12, 3),
    ([1] * 9, [64, 1, 63, 65, 128, 700, 0, 129, 400], 64, 8),
    ([2, 0, 1] * 9, [300, 40, 64] * 9, 20, 5),
    ([1] * 38, list(range(5, 195, 5)), 8, 8),
    ([1] * 39, list(range(5, 200, 5)), 8, 8),
]


@pytest.mark.parametrize("dtype,dim", [(BF, 128), (FP, 64)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (64, 3), (130, 70)])
@pytest.mark.parametrize("units", range(len(UNITS)))
def test_shared_and_cut_units(units, window, sinks, dtype, dim):
    b = Batch(*UNITS[units], dim, dtype, seed=300 + units)
    want = b.reference(window=window, sinks=sinks)
    b.check(b.attend(window=window, sinks=sinks), want)
    b.check(_wide(b).attend(window=window, sinks=sinks), want)


@pytest.mark.parametrize("heads,kv,dim", [(8, 2, 128), (40, 1, 64)])
def test_a_hint_too_small_changes_nothing_but_speed(heads, kv, dim):
    """Requests of more rows than a block holds, called as single tokens."""
    b = Batch([40, 1, 0, 7], [120, 90, 30, 3], heads, kv, dim, BF, seed=320)
    b.check(b.attend(max_query_len=1), b.reference())


@pytest.mark.parametrize("dtype", [BF, FP])
def test_nonfinite_values_reach_only_rows_that_see_them(dtype):
    b = Batch([4, 1], [130, 200], 8, 2, 64, dtype, seed=321)
    clean, _ = b.attend(window=70, sinks=2)
    for key, value in ((129, float("nan")), (127, float("inf")), (58, float("-inf"))):
        page, slot = int(b.table[0, key // 64]), key % 64
        keep = b.v[page, slot].clone()
        b.v[page, slot] = value
        out, _ = b.attend(window=70, sinks=2)
        b.v[page, slot] = keep
        pos = torch.arange(4, device=DEV) + 126
        rows = torch.ones(5, dtype=torch.bool, device=DEV)
        rows[:4] = ~((key <= pos) & ((pos - key < 70) | (key < 2)))
        assert torch.equal(out[rows], clean[rows])
        assert not torch.isfinite(out[~rows]).any()


def test_results_do_not_depend_on_timing():
    b = Batch([1] * 6, [900, 3, 400, 64, 1000, 5], 16, 2, 128, BF, seed=322)
    idx = _lists(b, 300)
    first, listed = b.attend(), b.attend_selected(idx)
    for _ in range(5):
        for again, want in ((b.attend(), first), (b.attend_selected(idx), listed)):
            assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


# tokens of one request over 900 keys, heads, kv heads, list length: clusters of 8, 4, 2 and 1 blocks,
# empty rows among them; then more units than clusters take, and rows of two blocks of 16
@pytest.mark.parametrize("tokens,heads,kv,topk", [(1, 4, 1, 2000), (5, 16, 8, 512), (9, 32, 16, 300), (30, 10, 5, 700),
                                                  (38, 8, 8, 130), (39, 8, 8, 800), (20, 40, 2, 700)])
@pytest.mark.parametrize("dtype,dim", [(BF, 64), (FP, 128)])
def test_lists_of_few_tokens(tokens, heads, kv, topk, dtype, dim):
    b = Batch([tokens], [900], heads, kv, dim, dtype, seed=330 + tokens)
    idx = _lists(b, topk, empty_rows=(0, 3))
    b.check(b.attend_selected(idx), b.reference(indices=idx))


def test_given_outputs_and_a_captured_step():
    b = Batch([1, 2], [500, 70], 8, 2, 128, BF, seed=340)
    want = b.reference()
    out, lse = torch.full_like(b.q, 7.0), torch.full((3, 8), 7.0, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        saib.indexer_attend_paged(b.q, b.k, b.v, b.table, b.lens, b.start, 2, out=out, lse=lse)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            saib.indexer_attend_paged(b.q, b.k, b.v, b.table, b.lens, b.start, 2, out=out, lse=lse)
        out.fill_(9.0)
        graph.replay()
    side.synchronize()
    b.check((out, lse), want)


def test_a_given_workspace_changes_nothing():
    b = Batch([1, 2], [500, 70], 8, 2, 128, BF, seed=341)
    idx = _lists(b, 200)
    ws = saib.attend_workspace(3, 2, 8, 2, 128, DEV)
    for a, c in ((b.attend(), b.attend(workspace=ws)),
                 (b.attend_selected(idx), b.attend_selected(idx, workspace=ws))):
        assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])
