"""Refusals of the paged-attention and page calls, on the CPU: the C entry
points reject bad arguments before they touch the device, and the binding
rejects tensors of a wrong type, shape, stride or device."""
import ctypes as C

import pytest
import torch

import sparse_attention_indexer_block_gb300 as saib
from sparse_attention_indexer_block_gb300 import binding
from sparse_attention_indexer_block_gb300 import build as libbuild

FAKE = 1 << 20  # an aligned non-null address; these calls fail before using it
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return saib.load()


def _args(**over):
    a = dict(q=FAKE, k=FAKE, v=FAKE, block_table=FAKE, seq_lens=FAKE, query_start_loc=FAKE,
             indices=FAKE, out=FAKE, lse=FAKE, workspace=FAKE, workspace_bytes=1 << 40,
             q_stride_token=1024, q_stride_head=128, k_stride_page=16384, k_stride_token=256,
             k_stride_head=128, v_stride_page=16384, v_stride_token=256, v_stride_head=128,
             num_pages=10, bt_stride=4, indices_stride=64, bt_width=4, num_reqs=2, num_tokens=6,
             num_heads=8, num_kv_heads=2, head_dim=128, dtype=0, max_query_len=3, window=0, sinks=0,
             topk=64, scale=0.1)
    a.update(over)
    return binding.Attend(**a)


COMMON = [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(out=None), INVALID), (dict(block_table=None), INVALID),
    (dict(query_start_loc=None), INVALID), (dict(workspace=None), INVALID),
    (dict(q=FAKE + 8), INVALID), (dict(k=FAKE + 2), INVALID), (dict(out=FAKE + 8), INVALID),
    (dict(workspace=FAKE + 128), INVALID), (dict(lse=FAKE + 2), INVALID),
    (dict(dtype=2), UNSUPPORTED), (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=256), UNSUPPORTED),
    (dict(num_heads=9), INVALID), (dict(num_heads=0), INVALID), (dict(num_kv_heads=0), INVALID),
    (dict(num_tokens=-1), INVALID), (dict(num_reqs=-1), INVALID),
    (dict(num_tokens=1 << 30), UNSUPPORTED),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID),
    (dict(num_pages=0), INVALID), (dict(bt_width=0), INVALID), (dict(bt_stride=3), INVALID),
    (dict(q_stride_head=4), INVALID), (dict(k_stride_token=-8), INVALID),
    (dict(v_stride_page=20), INVALID), (dict(workspace_bytes=64), WORKSPACE),
]


@pytest.mark.parametrize("over,status", COMMON)
def test_attend_refusals(lib, over, status):
    a = _args(**over)
    assert lib.indexer_attend_paged(C.byref(a), None) == status
    assert lib.indexer_attend_selected(C.byref(a), None) == status


def test_attend_refusals_of_one_form(lib):
    paged, selected = lib.indexer_attend_paged, lib.indexer_attend_selected
    assert paged(None, None) == INVALID and selected(None, None) == INVALID
    for over in (dict(window=-1), dict(sinks=-1), dict(max_query_len=-1), dict(seq_lens=None),
                 dict(seq_lens=FAKE + 2)):
        assert paged(C.byref(_args(**over)), None) == INVALID
    for over in (dict(topk=0), dict(indices_stride=63), dict(indices=None), dict(indices=FAKE + 2)):
        assert selected(C.byref(_args(**over)), None) == INVALID


def test_attend_of_nothing_is_accepted(lib):
    for over in (dict(num_tokens=0, q=None, out=None), dict(num_reqs=0, block_table=None)):
        assert lib.indexer_attend_paged(C.byref(_args(**over)), None) == OK
        assert lib.indexer_attend_selected(C.byref(_args(**over)), None) == OK


def test_attend_workspace_sizes(lib):
    n = C.c_size_t(0)
    f = lib.indexer_attend_workspace_bytes
    assert f(100, 4, 8, 2, 128, C.byref(n)) == OK
    small = n.value
    assert f(100000, 400, 8, 2, 128, C.byref(n)) == OK and n.value > small > 0
    assert f(100, 4, 8, 2, 128, None) == INVALID
    assert f(-1, 4, 8, 2, 128, C.byref(n)) == INVALID
    assert f(100, 4, 8, 3, 128, C.byref(n)) == INVALID
    assert f(100, 4, 8, 2, 80, C.byref(n)) == UNSUPPORTED
    assert f(1 << 30, 4, 8, 2, 128, C.byref(n)) == UNSUPPORTED


def _pool(**over):
    a = dict(base=FAKE, page_stride=8448, page_bytes=8448)
    a.update(over)
    return (binding.PagePool * 1)(binding.PagePool(**a))


BAD_POOLS = [dict(base=None), dict(base=FAKE + 8), dict(page_bytes=8440), dict(page_stride=8440),
             dict(page_bytes=0), dict(page_stride=8432)]


@pytest.mark.parametrize("over", BAD_POOLS)
def test_page_pool_refusals(lib, over):
    p = _pool(**over)
    assert lib.indexer_copy_pages(p, 1, 10, FAKE, FAKE, 3, None, None) == INVALID
    assert lib.indexer_fork_pages(p, 1, 10, FAKE, 4, 4, 3, FAKE, FAKE, FAKE, FAKE, 1, FAKE, FAKE, None,
                                  None) == INVALID
    assert lib.indexer_compact_pages(p, 1, 10, FAKE, 4, 4, 3, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 30,
                                     None, None) == INVALID


def test_page_call_refusals(lib):
    p = _pool()
    copy, fork = lib.indexer_copy_pages, lib.indexer_fork_pages
    free, compact = lib.indexer_free_pages, lib.indexer_compact_pages
    assert copy(p, 1, 0, FAKE, FAKE, 3, None, None) == INVALID
    assert copy(p, 1, 10, None, FAKE, 3, None, None) == INVALID
    assert copy(p, 1, 10, FAKE, FAKE, -1, None, None) == INVALID
    assert copy(p, -1, 10, FAKE, FAKE, 3, None, None) == INVALID
    assert copy(p, 1, 10, None, None, 0, None, None) == OK
    base = [p, 1, 10, FAKE, 4, 4, 3, FAKE, FAKE, FAKE, FAKE, 1, FAKE, FAKE, None, None]
    for at, value in ((3, None), (4, 3), (5, 0), (6, 0), (7, None), (8, None), (9, None), (10, None),
                      (11, 4), (11, -1), (12, None), (13, None), (8, FAKE + 2)):
        bad = list(base)
        bad[at] = value
        assert fork(*bad) == INVALID, at
    assert fork(*(base[:11] + [0] + base[12:])) == OK
    base = [FAKE, 4, 4, 3, FAKE, FAKE, 10, FAKE, 1, None, None]
    for at, value in ((0, None), (1, 3), (2, 0), (3, 0), (4, None), (5, None), (6, 0), (7, None), (8, 4),
                      (8, -1)):
        bad = list(base)
        bad[at] = value
        assert free(*bad) == INVALID, at
    base = [p, 1, 10, FAKE, 4, 4, 3, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 30, None, None]
    for at, value in ((2, 0), (3, None), (5, 0), (7, None), (8, None), (9, None), (10, None), (11, None),
                      (11, FAKE + 16)):
        bad = list(base)
        bad[at] = value
        assert compact(*bad) == INVALID, at
    bad = list(base)
    bad[12] = 16
    assert compact(*bad) == WORKSPACE
    n = C.c_size_t(0)
    assert lib.indexer_compact_workspace_bytes(0, C.byref(n)) == INVALID
    assert lib.indexer_compact_workspace_bytes(1000, C.byref(n)) == OK and n.value >= 8000


# ---- the binding -----------------------------------------------------------


def _tensors(**over):
    t = dict(q=torch.zeros(6, 8, 128, dtype=torch.bfloat16),
             k_cache=torch.zeros(10, 64, 2, 128, dtype=torch.bfloat16),
             v_cache=torch.zeros(10, 64, 2, 128, dtype=torch.bfloat16),
             block_table=torch.zeros(2, 4, dtype=torch.int32),
             seq_lens=torch.zeros(2, dtype=torch.int32),
             query_start_loc=torch.zeros(3, dtype=torch.int32))
    t.update(over)
    return t


BAD_TENSORS = [
    dict(q=torch.zeros(6, 8, 128)), dict(q=torch.zeros(6, 8, 64, dtype=torch.bfloat16)),
    dict(q=torch.zeros(6, 1024, dtype=torch.bfloat16)),
    dict(q=torch.zeros(6, 7, 128, dtype=torch.bfloat16)),
    dict(q=torch.zeros(6, 128, 8, dtype=torch.bfloat16).transpose(1, 2)),
    dict(k_cache=torch.zeros(10, 64, 2, 128, dtype=torch.float16)),
    dict(k_cache=torch.zeros(10, 32, 2, 128, dtype=torch.bfloat16)),
    dict(v_cache=torch.zeros(9, 64, 2, 128, dtype=torch.bfloat16)),
    dict(v_cache=torch.zeros(10, 64, 128, 2, dtype=torch.bfloat16).transpose(2, 3)),
    dict(block_table=torch.zeros(2, 4, dtype=torch.int64)),
    dict(block_table=torch.zeros(3, 4, dtype=torch.int32)),
    dict(block_table=torch.zeros(2, 0, dtype=torch.int32)),
    dict(block_table=torch.zeros(4, 2, dtype=torch.int32).t()),
    dict(seq_lens=torch.zeros(3, dtype=torch.int32)), dict(seq_lens=torch.zeros(2)),
    dict(query_start_loc=torch.zeros(0, dtype=torch.int32)),
    dict(query_start_loc=torch.zeros(3, 1, dtype=torch.int32)),
    dict(out=torch.zeros(6, 8, 128)), dict(lse=torch.zeros(6, 4)),
    dict(dev_error=torch.zeros(1, dtype=torch.int64)),
    dict(),  # all well but on the CPU
    dict(window=-1), dict(window=1 << 31), dict(sinks=-5), dict(max_query_len=1 << 40),
]


@pytest.mark.parametrize("over", BAD_TENSORS)
def test_binding_refuses_tensors(over):
    with pytest.raises(saib.IndexerError):
        saib.indexer_attend_paged(**_tensors(**over))
    if not {"seq_lens", "window", "sinks", "max_query_len"} & set(over):
        t = _tensors(**over)
        t.pop("seq_lens")
        with pytest.raises(saib.IndexerError):
            saib.indexer_attend_selected(indices=torch.zeros(6, 16, dtype=torch.int32), **t)


def test_binding_refuses_lists():
    t = _tensors()
    t.pop("seq_lens")
    for indices in (None, torch.zeros(5, 16, dtype=torch.int32), torch.zeros(6, 16),
                    torch.zeros(6, 0, dtype=torch.int32)):
        with pytest.raises(saib.IndexerError):
            saib.indexer_attend_selected(indices=indices, **t)


def test_binding_refuses_page_tensors():
    i32 = dict(dtype=torch.int32)
    pool, table, lens, refs = (torch.zeros(10, 64), torch.zeros(3, 4, **i32), torch.zeros(3, **i32),
                               torch.zeros(10, **i32))
    rows = torch.zeros(1, **i32)
    calls = [
        lambda: saib.indexer_copy_pages([pool], rows, rows),                  # on the CPU
        lambda: saib.indexer_copy_pages([], rows, rows),
        lambda: saib.indexer_copy_pages([pool], rows, torch.zeros(2, **i32)),
        lambda: saib.indexer_copy_pages([pool], rows.long(), rows.long()),
        lambda: saib.indexer_copy_pages([torch.zeros(10, 3)], rows, rows),
        lambda: saib.indexer_copy_pages([torch.zeros(64, 10).t()], rows, rows),
        lambda: saib.indexer_copy_pages([pool, torch.zeros(9, 64)], rows, rows),
        lambda: saib.indexer_fork_pages([pool], table, lens, refs, rows, rows),
        lambda: saib.indexer_fork_pages([pool], table, lens, torch.zeros(9, **i32), rows, rows),
        lambda: saib.indexer_fork_pages([pool], table.long(), lens, refs, rows, rows),
        lambda: saib.indexer_free_pages(table, lens, refs, rows),
        lambda: saib.indexer_free_pages(table, lens[:2], refs, rows),
        lambda: saib.indexer_compact_pages([pool], table, lens, refs),
        lambda: saib.indexer_compact_pages([pool], table, lens, refs, remap=torch.zeros(4, **i32)),
    ]
    for call in calls:
        with pytest.raises(saib.IndexerError):
            call()


def test_a_call_that_needs_a_workspace_says_so(lib):
    """A null workspace of 0 bytes: refused before any work unless the call needs none."""
    none = dict(workspace=None, workspace_bytes=0)
    assert lib.indexer_attend_paged(C.byref(_args(max_query_len=100, **none)), None) == WORKSPACE
    assert lib.indexer_attend_paged(C.byref(_args(num_reqs=5000, num_tokens=5000, **none)), None) == WORKSPACE
    assert lib.indexer_attend_paged(C.byref(_args(bt_width=4000, bt_stride=4000, **none)), None) == WORKSPACE
    assert lib.indexer_attend_selected(C.byref(_args(num_tokens=5000, **none)), None) == WORKSPACE
