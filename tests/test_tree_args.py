"""Refusals of the append, MXFP4 insert and tree calls, on the CPU: the C entry points reject bad
arguments before they touch the device, and the binding rejects tensors of a wrong type, shape, stride or
device."""
import ctypes as C

import pytest
import torch

import sparse_attention_indexer_block_gb300 as saib
from sparse_attention_indexer_block_gb300 import binding
from sparse_attention_indexer_block_gb300 import build as libbuild
from test_serving_args import COMMON, FAKE, INVALID, OK, UNSUPPORTED, WORKSPACE, _args


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return saib.load()


def _append(**over):
    a = dict(q=FAKE, k=FAKE, v=FAKE, slot_mapping=FAKE, positions=FAKE, rotary=FAKE, q_out=FAKE, k_cache=FAKE,
             v_cache=FAKE, q_stride_token=1024, q_stride_head=128, k_stride_token=256, k_stride_head=128,
             v_stride_token=256, v_stride_head=128, q_out_stride_token=1024, q_out_stride_head=128,
             k_cache_stride_page=16384, k_cache_stride_token=256, k_cache_stride_head=128,
             v_cache_stride_page=16384, v_cache_stride_token=256, v_cache_stride_head=128, num_pages=10,
             num_positions=100, rotary_stride=128, num_tokens=0, num_heads=8, num_kv_heads=2, head_dim=128, dtype=0,
             rotary_dim=128, interleaved=0)
    a.update(over)
    return binding.Append(**a)


# (before the sizes of nothing to do, and after them)
@pytest.mark.parametrize("over,status", [
    (dict(dtype=2), UNSUPPORTED), (dict(head_dim=96), UNSUPPORTED), (dict(num_tokens=-1), INVALID),
    (dict(num_kv_heads=0), INVALID), (dict(num_heads=0), INVALID), (dict(num_pages=0), INVALID),
    (dict(num_pages=1 << 32), INVALID), (dict(num_heads=(1 << 20) + 1), UNSUPPORTED), (dict(num_tokens=1 << 29), UNSUPPORTED),
    (dict(rotary_dim=8), UNSUPPORTED), (dict(rotary_dim=72), UNSUPPORTED), (dict(rotary_dim=144), UNSUPPORTED),
    (dict(interleaved=2), INVALID), (dict(num_positions=0), INVALID), (dict(rotary_stride=64), INVALID),
    (dict(rotary_stride=130), INVALID), (dict(rotary=FAKE + 4), INVALID)])
def test_append_refusals_of_any_size(lib, over, status):
    assert lib.indexer_append_kv(C.byref(_append(**over)), None) == status


@pytest.mark.parametrize("over", [
    dict(k=None), dict(v=None), dict(slot_mapping=None), dict(positions=None), dict(k_cache=None), dict(v_cache=None),
    dict(q_out=None), dict(k=FAKE + 8), dict(v=FAKE + 2), dict(q=FAKE + 8), dict(q_out=FAKE + 8),
    dict(k_cache=FAKE + 8), dict(v_cache=FAKE + 8), dict(slot_mapping=FAKE + 4), dict(positions=FAKE + 2),
    dict(q_stride_token=4), dict(q_stride_head=-8), dict(q_out_stride_head=12), dict(q_out_stride_token=-8),
    dict(k_stride_token=4), dict(k_stride_head=4), dict(v_stride_token=4), dict(v_stride_head=-8),
    dict(k_cache_stride_page=4), dict(k_cache_stride_token=4), dict(k_cache_stride_head=4),
    dict(v_cache_stride_page=4), dict(v_cache_stride_token=4), dict(v_cache_stride_head=4)])
def test_append_refusals(lib, over):
    assert lib.indexer_append_kv(C.byref(_append(num_tokens=3, **over)), None) == INVALID


def test_append_of_nothing_is_accepted(lib):
    assert lib.indexer_append_kv(None, None) == INVALID
    assert lib.indexer_append_kv(C.byref(_append(k=None, q=None)), None) == OK
    assert lib.indexer_append_kv(C.byref(_append(rotary=None, rotary_dim=7, num_positions=0)), None) == OK


def test_insert_mxfp4_refusals(lib):
    f = lib.indexer_insert_keys_mxfp4
    base = [FAKE, 128, FAKE, 4, 128, FAKE, 8, FAKE, None, None]

    def call(at, value):
        return f(*base[:at], value, *base[at + 1:])

    for at, value in ((0, None), (0, FAKE + 8), (1, 120), (1, 132), (2, None), (2, FAKE + 4), (3, -1), (5, None),
                      (5, FAKE + 8), (6, -1), (7, FAKE + 8)):
        assert call(at, value) == INVALID, (at, value)
    assert call(4, 64) == UNSUPPORTED
    assert call(3, 0) == OK


@pytest.mark.parametrize("over,status", COMMON)
def test_attend_tree_refuses_what_the_paged_form_refuses(lib, over, status):
    assert lib.indexer_attend_tree(C.byref(_args(**over)), FAKE, 2, 2, FAKE, None) == status


def test_attend_tree_refusals(lib):
    f = lib.indexer_attend_tree
    assert f(None, FAKE, 2, 2, FAKE, None) == INVALID
    for over in (dict(window=-1), dict(sinks=-1), dict(max_query_len=-1), dict(seq_lens=None), dict(seq_lens=FAKE + 2)):
        assert f(C.byref(_args(**over)), FAKE, 2, 2, FAKE, None) == INVALID
    a = C.byref(_args(window=5, workspace_bytes=64))
    for masks, stride, words, positions in ((None, 2, 2, FAKE), (FAKE + 2, 2, 2, FAKE), (FAKE, 1, 2, FAKE),
                                            (FAKE, 2, 0, FAKE), (FAKE, 2, 2, None), (FAKE, 2, 2, FAKE + 2)):
        assert f(a, masks, stride, words, positions, None) == INVALID
    # (valid up to the workspace's size)
    assert f(a, FAKE, 2, 2, FAKE, None) == WORKSPACE
    assert f(C.byref(_args(workspace_bytes=64)), FAKE, 2, 2, None, None) == WORKSPACE
    for over in (dict(num_tokens=0, q=None, out=None), dict(num_reqs=0, block_table=None)):
        assert f(C.byref(_args(**over)), None, 2, 2, None, None) == OK


def test_plan_tree_refusals(lib):
    f = lib.indexer_plan_tree
    base = [FAKE, FAKE, FAKE, 2, 6, 0, 0, FAKE, 1, FAKE, FAKE, 4, None, None]

    def call(*changes):
        a = list(base)
        for at, value in changes:
            a[at] = value
        return f(*a)

    for at, value in ((0, None), (1, None), (2, None), (3, -1), (4, -1), (5, -1), (6, -1), (7, None), (8, 0), (9, None),
                      (11, 0), (11, -1), (0, FAKE + 2), (7, FAKE + 2), (9, FAKE + 1), (10, FAKE + 2)):
        assert call((at, value)) == INVALID, (at, value)
    assert call((3, 0)) == OK and call((4, 0), (0, None)) == OK


def _token_pool(**over):
    a = dict(base=FAKE, page_stride=16384, token_stride=256, piece_stride=0, pieces=1, piece_bytes=256)
    a.update(over)
    return (binding.TokenPool * 1)(binding.TokenPool(**a))


def test_commit_tree_refusals(lib):
    f = lib.indexer_commit_tree
    base = [_token_pool(), 1, 10, FAKE, 4, 4, 2, FAKE, FAKE, FAKE, 8, 8, FAKE, None, None]

    def call(at, value):
        return f(*base[:at], value, *base[at + 1:])

    for over in (dict(base=None), dict(base=FAKE + 2), dict(pieces=0), dict(piece_bytes=0), dict(piece_bytes=6),
                 dict(page_stride=-4), dict(page_stride=2), dict(token_stride=-4), dict(token_stride=6),
                 dict(piece_stride=-4), dict(piece_stride=2), dict(pieces=1 << 24, piece_bytes=1 << 10)):
        assert call(0, _token_pool(**over)) == INVALID, over
    two = (binding.TokenPool * 2)(*_token_pool(), *_token_pool())
    assert f(two, 2, *base[2:]) == INVALID                       # the same pool twice
    for at, value in ((0, None), (1, -1), (2, 0), (2, 1 << 31), (3, None), (4, 3), (5, 0), (6, -1), (7, None), (8, None),
                      (9, None), (10, 7), (11, -1), (3, FAKE + 2), (9, FAKE + 1), (12, FAKE + 2)):
        assert call(at, value) == INVALID, (at, value)
    assert call(6, 0) == OK


def _refused(status, call, *args, **kw):
    with pytest.raises(saib.IndexerError) as e:
        call(*args, **kw)
    assert e.value.status == status, str(e.value)


BF = torch.bfloat16


def _i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_binding_append_refusals():
    call = saib.indexer_append_kv
    k, v = torch.zeros((5, 2, 64), dtype=BF), torch.zeros((5, 2, 64), dtype=BF)
    kc, vc = torch.zeros((4, 64, 2, 64), dtype=BF), torch.zeros((4, 64, 2, 64), dtype=BF)
    slots, q, pos, rot = torch.zeros(5, dtype=torch.int64), torch.zeros((5, 4, 64), dtype=BF), _i32(5), torch.zeros((9, 32))
    full = dict(q=q, positions=pos, rotary=rot)
    for args in ((k[0], v, kc, vc, slots), (k, v[:4], kc, vc, slots), (k, v, kc[:, :, :1], vc, slots),
                 (k, v, kc, vc[:3], slots), (k, v.half(), kc, vc, slots), (k, v, kc, vc, slots.int()),
                 (k, v, kc, vc, slots[:4]), (k, v, kc, vc, torch.zeros(10, dtype=torch.int64)[::2]),
                 (torch.zeros((5, 2, 128), dtype=BF)[:, :, ::2], v, kc, vc, slots),
                 (k, v, torch.zeros((4, 64, 1, 64), dtype=BF).expand(4, 64, 2, 64), vc, slots)):
        _refused(INVALID, call, *args, **full)
    for args in ((k.float(), v, kc, vc, slots), (k, v, kc[:, :32], vc[:, :32], slots),
                 (k[..., :32], v[..., :32], kc[..., :32], vc[..., :32], slots)):
        _refused(UNSUPPORTED, call, *args, **full)
    for over in (dict(rotary=None), dict(positions=None), dict(positions=pos.long()), dict(positions=pos[:4]), dict(q=q[:4]),
                 dict(q=q.float()), dict(q=q[:, :0]), dict(rotary=rot.half()), dict(rotary=rot[0]),
                 dict(q_out=q.float()), dict(q_out=q[:, :2]), dict(q=None, q_out=q), dict(dev_error=torch.zeros(1, dtype=torch.int64)),
                 dict(q_out=torch.zeros((5, 1, 64), dtype=BF).expand(5, 4, 64))):
        _refused(INVALID, call, k, v, kc, vc, slots, **{**full, **over})
    for dim in (24, 80, 8):
        _refused(UNSUPPORTED, call, k, v, kc, vc, slots, **{**full, "rotary": torch.zeros((9, dim))})
    _refused(INVALID, call, k, v, kc, vc, slots, **full)   # not on a CUDA device


def test_binding_insert_mxfp4_refusals():
    call = saib.indexer_insert_keys_mxfp4
    k, slots, cache = torch.zeros((5, 128), dtype=BF), torch.zeros(5, dtype=torch.int64), torch.zeros((3, 4352), dtype=torch.uint8)
    for args, kw in (((k.float(), slots, cache), {}), ((k[0], slots, cache), {}), ((k, slots[:4], cache), {}),
                     ((k, slots.int(), cache), {}), ((k, slots, cache[:, :4351]), {}), ((k, slots, cache.int()), {}),
                     ((k, slots, torch.zeros((3, 8448), dtype=torch.uint8)), {}),
                     ((k, slots, torch.zeros((6, 4352), dtype=torch.uint8)[::2]), {}), ((k, slots, cache), dict(values=k.float())),
                     ((k, slots, cache), dict(values=k[:4])), ((k, slots, cache), {})):
        _refused(INVALID, call, *args, **kw)
    _refused(UNSUPPORTED, call, k[:, :64], slots, cache)


def test_binding_tree_refusals():
    q, cache = torch.zeros((6, 4, 64), dtype=BF), torch.zeros((3, 64, 2, 64), dtype=BF)
    base = [q, cache, cache, _i32(2, 4), _i32(2), _i32(3), _i32(6, 1)]
    for kw in (dict(window=3), dict(window=3, positions=_i32(5)), dict(positions=_i32(6).long()), dict(window=-1), {}):
        _refused(INVALID, saib.indexer_attend_tree, *base, **kw)
    for masks in (None, _i32(6, 0), _i32(5, 1), _i32(6), _i32(6, 1).long(), _i32(1, 2).expand(6, 2)):
        _refused(INVALID, saib.indexer_attend_tree, *base[:6], masks)

    base = [_i32(6), _i32(2), _i32(3), 6]
    for at, value in ((0, _i32(6).long()), (0, _i32(2, 3)), (1, _i32(3)), (2, _i32(0)), (2, _i32(4)), (3, 0), (3, -1)):
        _refused(INVALID, saib.indexer_plan_tree, *base[:at], value, *base[at + 1:])
    for kw in (dict(window=-1), dict(sinks=-1), dict(max_path=-1), dict(masks=_i32(6, 2)), dict(masks=_i32(1, 6).t()[:, :0]),
               dict(positions=_i32(5)), dict(paths=_i32(6, 3)), dict(paths=_i32(6, 3), max_path=4), {}):
        _refused(INVALID, saib.indexer_plan_tree, *base, **kw)


def test_binding_commit_refusals():
    cache = torch.zeros((3, 64, 2, 64), dtype=BF)
    index, mx = torch.zeros((3, 8448), dtype=torch.uint8), torch.zeros((3, 4352), dtype=torch.uint8)
    base = [[cache, index, mx], _i32(2, 4), _i32(2), _i32(3), _i32(2, 5)]
    for pools in ([cache[0, 0, 0]], [cache, index[:2]], [None], [cache.expand(3, 64, 2, 64)[:0]],
                  [torch.zeros((3, 64, 3), dtype=torch.uint8)], [torch.zeros((3, 64, 1, 64), dtype=BF).expand(3, 64, 2, 64)],
                  [torch.zeros((3, 64, 4, 2, 64), dtype=BF)[:, :, :, :1, :32].transpose(2, 3).expand(3, 64, 1, 4, 32)[..., ::2]],
                  [torch.zeros((3, 8450), dtype=torch.uint8)[:, :8448]]):
        _refused(INVALID, saib.indexer_commit_tree, pools, *base[1:])
    _refused(UNSUPPORTED, saib.indexer_commit_tree, [cache[:, :32]], *base[1:])
    for at, value in ((1, _i32(3, 4)), (1, _i32(2, 0)), (2, _i32(3)), (2, _i32(2).long()), (3, _i32(0)), (3, _i32(4)), (4, _i32(3, 5)),
                      (4, _i32(1, 5).expand(2, 5)), (4, _i32(2, 5).long())):
        _refused(INVALID, saib.indexer_commit_tree, *base[:at], value, *base[at + 1:])
    _refused(INVALID, saib.indexer_commit_tree, *base, ref_counts=_i32(4))
    _refused(INVALID, saib.indexer_commit_tree, [], *base[1:])
    _refused(INVALID, saib.indexer_commit_tree, *base)      # not on a CUDA device


def test_token_pools_of_strided_caches():
    """Head-major caches, halves of one array, whole tokens: what the binding makes of them."""
    def entries(*pools):
        return binding._native().token_pools(pools)

    plain = torch.zeros((3, 64, 2, 64), dtype=BF)
    heads = torch.zeros((3, 2, 64, 64), dtype=BF).transpose(1, 2)
    joint = torch.zeros((3, 2, 64, 2, 64), dtype=BF)
    assert entries(plain) == [(16384, 256, 256, 1, 256)]
    assert entries(heads) == [(16384, 128, 8192, 2, 128)]
    assert entries(joint[:, 0], joint[:, 1]) == [(32768, 256, 256, 1, 256)] * 2
    assert entries(torch.zeros((3, 8448), dtype=torch.uint8)) == [(8448, 128, 0, 1, 128), (8448, 4, 0, 1, 4)]
    assert entries(torch.zeros((3, 4352), dtype=torch.uint8)) == [(4352, 68, 0, 1, 68)]
    assert entries(torch.zeros((3, 64), dtype=torch.float32)) == [(256, 4, 4, 1, 4)]
