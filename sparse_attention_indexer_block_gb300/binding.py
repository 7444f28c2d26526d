"""Thin ctypes binding of the indexer's C ABI (``include/indexer.h``).

Argument marshalling only: every function forwards torch tensors' device
pointers, sizes and the current CUDA stream to the function of the same name
in ``libsaib.so`` and raises :class:`IndexerError` on a non-OK status. Torch is
used for device memory (outputs and workspaces the caller did not pass) and
streams. There is no fallback: without the built library every call raises.
The calls that run once a layer and step (attention, appends, trees) are
marshalled by a native module (``_marshal.so``, ``csrc/marshal.cpp``).
"""
from __future__ import annotations

import ctypes as C
import functools
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsaib.so")

IDX_OK = 0
STATUS_NAMES = {0: "IDX_OK", 1: "IDX_ERR_INVALID_ARG", 2: "IDX_ERR_UNSUPPORTED",
                3: "IDX_ERR_WORKSPACE", 4: "IDX_ERR_CUDA", 5: "IDX_ERR_CAPACITY"}
DEV_BAD_BLOCK, DEV_BAD_LEN, DEV_TIMEOUT, DEV_OVERFLOW = 1, 2, 4, 8
DEV_BAD_ROW, DEV_NO_PAGE, DEV_BAD_REF = 32, 64, 128
NUM_HEADS, HEAD_DIM, PAGE_TOKENS, PAGE_BYTES, MAX_TOPK = 64, 128, 64, 8448, 2048
MXFP4_PAGE_BYTES, MXFP4_TOKEN_BYTES = 4352, 68
DCP_MAX_CANDIDATES = 16384


class Attend(C.Structure):
    """idx_attend of indexer.h."""
    _fields_ = ([(n, C.c_void_p) for n in ("q", "k", "v", "block_table", "seq_lens",
                                           "query_start_loc", "indices", "out", "lse",
                                           "workspace")]
                + [("workspace_bytes", C.c_size_t), ("dev_error", C.c_void_p)]
                + [(n, C.c_int64) for n in ("q_stride_token", "q_stride_head", "k_stride_page",
                                            "k_stride_token", "k_stride_head", "v_stride_page",
                                            "v_stride_token", "v_stride_head", "num_pages",
                                            "bt_stride", "indices_stride")]
                + [(n, C.c_int32) for n in ("bt_width", "num_reqs", "num_tokens", "num_heads",
                                            "num_kv_heads", "head_dim", "dtype", "max_query_len",
                                            "window", "sinks", "topk")]
                + [("scale", C.c_float)])


class PagePool(C.Structure):
    """idx_page_pool of indexer.h."""
    _fields_ = [("base", C.c_void_p), ("page_stride", C.c_int64), ("page_bytes", C.c_int64)]


class Append(C.Structure):
    """idx_append of indexer.h."""
    _fields_ = ([(n, C.c_void_p) for n in ("q", "k", "v", "slot_mapping", "positions", "rotary", "q_out",
                                           "k_cache", "v_cache", "dev_error")]
                + [(n, C.c_int64) for n in ("q_stride_token", "q_stride_head", "k_stride_token",
                                            "k_stride_head", "v_stride_token", "v_stride_head",
                                            "q_out_stride_token", "q_out_stride_head",
                                            "k_cache_stride_page", "k_cache_stride_token",
                                            "k_cache_stride_head", "v_cache_stride_page",
                                            "v_cache_stride_token", "v_cache_stride_head",
                                            "num_pages", "num_positions", "rotary_stride")]
                + [(n, C.c_int32) for n in ("num_tokens", "num_heads", "num_kv_heads", "head_dim",
                                            "dtype", "rotary_dim", "interleaved")])


class TokenPool(C.Structure):
    """idx_token_pool of indexer.h."""
    _fields_ = [("base", C.c_void_p), ("page_stride", C.c_int64), ("token_stride", C.c_int64),
                ("piece_stride", C.c_int64), ("pieces", C.c_int32), ("piece_bytes", C.c_int32)]


# exported symbols and their ctypes signatures (kept in step with indexer.h)
_P, _I32, _I64, _SZ = C.c_void_p, C.c_int32, C.c_int64, C.c_size_t
SIGNATURES = {
    "indexer_status_string": (C.c_char_p, [C.c_int]),
    "indexer_last_cuda_error": (C.c_char_p, []),
    "indexer_expand_decode_rows": (C.c_int, [_P, _P, _I32, _I32, _P, _I64, _I32, _I32, _P, _P,
                                             _I64, _I64, _P, _P]),
    "indexer_quantize_q": (C.c_int, [_P, _P, _I64, _I32, _I32, _P, _P, _P]),
    "indexer_insert_keys": (C.c_int, [_P, _P, _I64, _I32, _P, _I64, _P, _P]),
    "indexer_decode_workspace_bytes": (C.c_int, [_I32, _I32, _I32, C.POINTER(_SZ)]),
    "indexer_decode_topk": (C.c_int, [_P, _P, _P, _I64, _P, _I64, _I32, _P, _I32, _I32, _I32,
                                      _I32, _I32, _P, _P, _SZ, _P, _P]),
    "indexer_decode_topk_from_lens": (C.c_int, [_P, _P, _P, _I64, _P, _I64, _I32, _P, _P, _I32,
                                                _I32, _I32, _I32, _I32, _P, _P, _SZ, _P, _P]),
    "indexer_decode_logits": (C.c_int, [_P, _P, _P, _I64, _P, _I64, _I32, _P, _I32, _I32, _I32,
                                        _I32, _I32, _P, _I64, _P, _SZ, _P, _P]),
    "indexer_plan_prefill_chunks": (C.c_int, [_P, _P, _I32, _I64, _I64, _P, _I32,
                                              C.POINTER(_I32)]),
    "indexer_prefill_workspace_bytes": (C.c_int, [_P, _P, _I32, _I32, _I64, _I64,
                                                  C.POINTER(_SZ)]),
    "indexer_prefill_topk": (C.c_int, [_P, _P, _P, _I64, _P, _I64, _I32, _P, _P, _P, _P, _I32,
                                       _I32, _I32, _I32, _I64, _I64, _P, _P, _SZ, _P, _P]),
    "indexer_profile_events": (C.c_int, [_P, _P]),
    "indexer_trace_buffer": (C.c_int, [_P, _SZ]),
    "indexer_debug_wait_limit": (C.c_int, [C.c_uint64, _I32]),
    "indexer_debug_divide": (C.c_int, [_P, _P, _I64, _P, _P, _P]),
    "indexer_debug_decode_plan": (C.c_int, [_I32, _I32, _I32, C.POINTER(_I64),
                                            C.POINTER(_I32), C.POINTER(_I32)]),
    "indexer_decode_topk_noalloc": (C.c_int, [_P, _P, _P, _I64, _P, _I64, _I32, _P, _I32, _I32,
                                              _I32, _I32, _I32, _P, _P, _P]),
    "indexer_index_key_counts": (C.c_int, [_P, _I64, _I32, _I32, _I32, _I32, _P, _P]),
    "indexer_decode_topk_values": (C.c_int, [_P, _P, _P, _I64, _P, _I64, _I32, _P, _I32, _I32,
                                             _I32, _I32, _I32, _I32, _I32, _I32, _I32, _P, _P, _P,
                                             _SZ, _P, _P]),
    "indexer_prefill_topk_values": (C.c_int, [_P, _P, _P, _I64, _P, _I64, _I32, _P, _P, _P, _P,
                                              _I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32,
                                              _I64, _I64, _P, _P, _P, _SZ, _P, _P]),
    "indexer_dcp_merge": (C.c_int, [_P, _P, _I32, _I64, _I32, _P, _P, _P]),
    "indexer_block_topk": (C.c_int, [_P, _I64, _P, _I64, _I32, _I32, _I32, _I32, _P, _I32, _P,
                                     _P]),
    "indexer_expand_pools": (C.c_int, [_P, _I32, _P, _P, _I64, _I32, _P, _I32, _P, _P]),
    "indexer_decode_topk_mxfp4": (C.c_int, [_P, _P, _P, _I64, _P, _I64, _I32, _P, _I32, _I32,
                                            _I32, _I32, _I32, _P, _P, _SZ, _P, _P]),
    "indexer_decode_logits_mxfp4": (C.c_int, [_P, _P, _P, _I64, _P, _I64, _I32, _P, _I32, _I32,
                                              _I32, _I32, _I32, _P, _I64, _P, _SZ, _P, _P]),
}

SIGNATURES.update({
    "indexer_attend_workspace_bytes": (C.c_int, [_I32, _I32, _I32, _I32, _I32, C.POINTER(_SZ)]),
    "indexer_attend_paged": (C.c_int, [_P, _P]),
    "indexer_attend_selected": (C.c_int, [_P, _P]),
    "indexer_copy_pages": (C.c_int, [C.POINTER(PagePool), _I32, _I64, _P, _P, _I32, _P, _P]),
    "indexer_fork_pages": (C.c_int, [C.POINTER(PagePool), _I32, _I64, _P, _I64, _I32, _I32, _P, _P,
                                     _P, _P, _I32, _P, _P, _P, _P]),
    "indexer_free_pages": (C.c_int, [_P, _I64, _I32, _I32, _P, _P, _I64, _P, _I32, _P, _P]),
    "indexer_compact_workspace_bytes": (C.c_int, [_I64, C.POINTER(_SZ)]),
    "indexer_compact_pages": (C.c_int, [C.POINTER(PagePool), _I32, _I64, _P, _I64, _I32, _I32, _P,
                                        _P, _P, _P, _P, _SZ, _P, _P]),
    "indexer_attend_tree": (C.c_int, [_P, _P, _I64, _I32, _P, _P]),
    "indexer_append_kv": (C.c_int, [_P, _P]),
    "indexer_insert_keys_mxfp4": (C.c_int, [_P, _I64, _P, _I64, _I32, _P, _I64, _P, _P, _P]),
    "indexer_plan_tree": (C.c_int, [_P, _P, _P, _I32, _I32, _I32, _I32, _P, _I32, _P, _P, _I32, _P,
                                    _P]),
    "indexer_commit_tree": (C.c_int, [_P, _I32, _I64, _P, _I64, _I32, _I32, _P, _P, _P, _I64, _I32,
                                      _P, _P, _P]),
})

_lock = threading.Lock()
_lib = _marshal = None


class IndexerError(RuntimeError):
    def __init__(self, fn: str, status: int, detail: str = ""):
        msg = f"{fn} failed: {STATUS_NAMES.get(status, status)}"
        super().__init__(msg + (f" ({detail})" if detail else ""))
        self.status = status


def load(path: str = LIB_PATH):
    """Loads libsaib.so (build it with ``build.build()`` first)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(f"indexer CUDA library not built ({path}); run "
                               "sparse_attention_indexer_block_gb300.build.build()")
        lib = C.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
        return lib


def _native():
    """The module of the calls of every layer, on the library that load() has loaded."""
    global _marshal
    if _marshal is None:
        lib = load()
        try:
            from . import _marshal as marshal
        except ImportError as e:
            raise RuntimeError(f"the native marshalling is not built for this Python and torch ({e}); run "
                               "sparse_attention_indexer_block_gb300.build.build()") from e
        marshal.set_error_class(IndexerError)
        marshal.bind(lib._handle)
        _marshal = marshal
    return _marshal


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return C.c_void_p(t)
    return C.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        return C.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return C.c_void_p(stream)
    return C.c_void_p(stream.cuda_stream)


def _check(name, st):
    if st != IDX_OK:
        detail = load().indexer_last_cuda_error().decode() if st == 4 else ""
        raise IndexerError(name, st, detail)


def _host_i32(t):
    import numpy as np
    if isinstance(t, torch.Tensor):
        t = t.detach().cpu().numpy()
    return np.ascontiguousarray(t, dtype=np.int32)


def indexer_status_string(status: int) -> str:
    return load().indexer_status_string(status).decode()


def indexer_expand_decode_rows(seq_lens, decode_lens, next_n: int, mode: int = 0,
                               block_table=None, row_seq_lens=None, row_block_table=None,
                               num_out_rows: int | None = None, want_block_table: bool = False,
                               dev_error=None, stream=None):
    R = int(seq_lens.shape[0])
    if num_out_rows is None:
        num_out_rows = R * next_n
    dev = seq_lens.device
    if row_seq_lens is None:
        row_seq_lens = torch.empty(num_out_rows, dtype=torch.int32, device=dev)
    W, bt_stride, out_stride = 0, 0, 0
    if block_table is not None:
        W = int(block_table.shape[1])
        bt_stride = int(block_table.stride(0))
        if row_block_table is None and want_block_table:
            row_block_table = torch.zeros((num_out_rows, W), dtype=torch.int32, device=dev)
        if row_block_table is not None:
            out_stride = int(row_block_table.stride(0))
    st = load().indexer_expand_decode_rows(
        _ptr(seq_lens), _ptr(decode_lens), R, next_n, _ptr(block_table), bt_stride, W, mode,
        _ptr(row_seq_lens), _ptr(row_block_table), out_stride, num_out_rows, _ptr(dev_error),
        _stream(stream))
    _check("indexer_expand_decode_rows", st)
    return row_seq_lens, row_block_table


def indexer_quantize_q(q, weights, q_fp8=None, weights_scaled=None, stream=None):
    rows = int(q.shape[0])
    if q_fp8 is None:
        q_fp8 = torch.empty((rows, NUM_HEADS, HEAD_DIM), dtype=torch.uint8, device=q.device)
    if weights_scaled is None:
        weights_scaled = torch.empty((rows, NUM_HEADS), dtype=torch.float32, device=q.device)
    st = load().indexer_quantize_q(_ptr(q), _ptr(weights), rows, int(q.shape[1]),
                                   int(q.shape[2]), _ptr(q_fp8), _ptr(weights_scaled),
                                   _stream(stream))
    _check("indexer_quantize_q", st)
    return q_fp8, weights_scaled


def indexer_insert_keys(k, slot_mapping, index_cache, dev_error=None, stream=None):
    """Quantises k (bf16 [T, 128]) per token and writes it into the paged
    index cache (uint8 [pages, 8448]) at slot_mapping (int64 [T]); in place."""
    st = load().indexer_insert_keys(_ptr(k), _ptr(slot_mapping), int(k.shape[0]), int(k.shape[1]),
                                    _ptr(index_cache), int(index_cache.shape[0]),
                                    _ptr(dev_error), _stream(stream))
    _check("indexer_insert_keys", st)
    return index_cache


def indexer_decode_workspace_bytes(num_reqs: int, next_n: int, topk: int) -> int:
    out = C.c_size_t(0)
    _check("indexer_decode_workspace_bytes",
           load().indexer_decode_workspace_bytes(num_reqs, next_n, topk, C.byref(out)))
    return int(out.value)


def decode_workspace(num_reqs: int, next_n: int, topk: int, device="cuda"):
    n = indexer_decode_workspace_bytes(num_reqs, next_n, topk)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def indexer_decode_topk(q, weights, index_cache, block_table, row_seq_lens, next_n: int,
                        topk: int = MAX_TOPK, out_idx=None, workspace=None, dev_error=None,
                        stream=None):
    R = int(block_table.shape[0])
    rows = R * next_n
    if out_idx is None:
        out_idx = torch.empty((rows, topk), dtype=torch.int32, device=q.device)
    if workspace is None:
        workspace = decode_workspace(R, next_n, topk, q.device)
    st = load().indexer_decode_topk(
        _ptr(q), _ptr(weights), _ptr(index_cache), int(index_cache.shape[0]), _ptr(block_table),
        int(block_table.stride(0)), int(block_table.shape[1]), _ptr(row_seq_lens), R, next_n,
        int(q.shape[1]), int(q.shape[2]), topk, _ptr(out_idx), _ptr(workspace),
        int(workspace.numel() * workspace.element_size()), _ptr(dev_error), _stream(stream))
    _check("indexer_decode_topk", st)
    return out_idx


def indexer_decode_topk_from_lens(q, weights, index_cache, block_table, seq_lens, decode_lens,
                                  next_n: int, topk: int = MAX_TOPK, out_idx=None,
                                  workspace=None, dev_error=None, stream=None):
    """indexer_decode_topk with the row expansion done on the device by the
    launch itself: seq_lens, decode_lens int32 [num_reqs]."""
    R = int(block_table.shape[0])
    rows = R * next_n
    if out_idx is None:
        out_idx = torch.empty((rows, topk), dtype=torch.int32, device=q.device)
    if workspace is None:
        workspace = decode_workspace(R, next_n, topk, q.device)
    st = load().indexer_decode_topk_from_lens(
        _ptr(q), _ptr(weights), _ptr(index_cache), int(index_cache.shape[0]), _ptr(block_table),
        int(block_table.stride(0)), int(block_table.shape[1]), _ptr(seq_lens), _ptr(decode_lens),
        R, next_n, int(q.shape[1]), int(q.shape[2]), topk, _ptr(out_idx), _ptr(workspace),
        int(workspace.numel() * workspace.element_size()), _ptr(dev_error), _stream(stream))
    _check("indexer_decode_topk_from_lens", st)
    return out_idx


def indexer_index_key_counts(row_seq_lens, compress_ratio: int = 1, dcp_rank: int = 0,
                             dcp_world: int = 1, dcp_interleave: int = 1, key_counts=None,
                             stream=None):
    """Cache entries each row sees on rank dcp_rank of a compressed and / or
    key-sharded cache (int32 tensors)."""
    n = int(row_seq_lens.numel())
    if key_counts is None:
        key_counts = torch.empty_like(row_seq_lens)
    st = load().indexer_index_key_counts(_ptr(row_seq_lens), n, compress_ratio, dcp_rank,
                                         dcp_world, dcp_interleave, _ptr(key_counts),
                                         _stream(stream))
    _check("indexer_index_key_counts", st)
    return key_counts


def indexer_decode_topk_values(q, weights, index_cache, block_table, row_seq_lens, next_n: int,
                               topk: int = MAX_TOPK, compress_ratio: int = 1, dcp_rank: int = 0,
                               dcp_world: int = 1, dcp_interleave: int = 1, out_idx=None,
                               out_val=None, workspace=None, dev_error=None, stream=None):
    """Top-k with the selected logits on one rank of a key-sharded cache
    (the whole cache when dcp_world == 1); indices in global positions.
    Returns (out_idx int32, out_val float32), both [rows, topk]."""
    R = int(block_table.shape[0])
    rows = R * next_n
    if out_idx is None:
        out_idx = torch.empty((rows, topk), dtype=torch.int32, device=q.device)
    if out_val is None:
        out_val = torch.empty((rows, topk), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = decode_workspace(R, next_n, topk, q.device)
    st = load().indexer_decode_topk_values(
        _ptr(q), _ptr(weights), _ptr(index_cache), int(index_cache.shape[0]), _ptr(block_table),
        int(block_table.stride(0)), int(block_table.shape[1]), _ptr(row_seq_lens), R, next_n,
        int(q.shape[1]), int(q.shape[2]), topk, compress_ratio, dcp_rank, dcp_world,
        dcp_interleave, _ptr(out_idx), _ptr(out_val), _ptr(workspace),
        int(workspace.numel() * workspace.element_size()), _ptr(dev_error), _stream(stream))
    _check("indexer_decode_topk_values", st)
    return out_idx, out_val


def indexer_dcp_merge(cand_val, cand_idx, topk: int = MAX_TOPK, out_idx=None, out_val=None,
                      stream=None):
    """The top k of the ranks' candidates cand_val float32 / cand_idx int32
    [world, rows, topk]. Returns (out_idx, out_val) [rows, topk]."""
    world, rows = int(cand_idx.shape[0]), int(cand_idx.shape[1])
    if out_idx is None:
        out_idx = torch.empty((rows, topk), dtype=torch.int32, device=cand_idx.device)
    st = load().indexer_dcp_merge(_ptr(cand_val), _ptr(cand_idx), world, rows, topk,
                                  _ptr(out_idx), _ptr(out_val), _stream(stream))
    _check("indexer_dcp_merge", st)
    return out_idx, out_val


def indexer_decode_topk_mxfp4(q, weights, index_cache, block_table, row_seq_lens,
                              topk: int = MAX_TOPK, out_idx=None, workspace=None, dev_error=None,
                              stream=None):
    """Decode top-k (next_n = 1) over an MXFP4 cache uint8 [pages, 4352]."""
    R = int(block_table.shape[0])
    if out_idx is None:
        out_idx = torch.empty((R, topk), dtype=torch.int32, device=q.device)
    if workspace is None:
        workspace = decode_workspace(R, 1, topk, q.device)
    st = load().indexer_decode_topk_mxfp4(
        _ptr(q), _ptr(weights), _ptr(index_cache), int(index_cache.shape[0]), _ptr(block_table),
        int(block_table.stride(0)), int(block_table.shape[1]), _ptr(row_seq_lens), R, 1,
        int(q.shape[1]), int(q.shape[2]), topk, _ptr(out_idx), _ptr(workspace),
        int(workspace.numel() * workspace.element_size()), _ptr(dev_error), _stream(stream))
    _check("indexer_decode_topk_mxfp4", st)
    return out_idx


def indexer_decode_logits_mxfp4(q, weights, index_cache, block_table, row_seq_lens,
                                topk: int = MAX_TOPK, out_logits=None, workspace=None,
                                dev_error=None, stream=None):
    R = int(block_table.shape[0])
    ld = int(block_table.shape[1]) * PAGE_TOKENS
    if out_logits is None:
        out_logits = torch.full((R, ld), float("nan"), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = decode_workspace(R, 1, topk, q.device)
    st = load().indexer_decode_logits_mxfp4(
        _ptr(q), _ptr(weights), _ptr(index_cache), int(index_cache.shape[0]), _ptr(block_table),
        int(block_table.stride(0)), int(block_table.shape[1]), _ptr(row_seq_lens), R, 1,
        int(q.shape[1]), int(q.shape[2]), topk, _ptr(out_logits), ld, _ptr(workspace),
        int(workspace.numel() * workspace.element_size()), _ptr(dev_error), _stream(stream))
    _check("indexer_decode_logits_mxfp4", st)
    return out_logits


def indexer_block_topk(logits, row_lens, block_size: int, topk_blocks: int, init_blocks: int = 0,
                       local_blocks: int = 0, out_cap: int | None = None, out=None, cnt=None,
                       stream=None):
    """Selected blocks per row (ascending, -1 after) and their counts."""
    rows = int(logits.shape[0])
    cap = out_cap or (topk_blocks + init_blocks + local_blocks)
    if out is None:
        out = torch.empty((rows, cap), dtype=torch.int32, device=logits.device)
    if cnt is None:
        cnt = torch.empty(rows, dtype=torch.int32, device=logits.device)
    st = load().indexer_block_topk(_ptr(logits), int(logits.stride(0)), _ptr(row_lens), rows,
                                   block_size, topk_blocks, init_blocks, local_blocks, _ptr(out),
                                   cap, _ptr(cnt), _stream(stream))
    _check("indexer_block_topk", st)
    return out, cnt


def indexer_expand_pools(pools, row_lens, pool_size: int, out_cap: int, pool_counts=None,
                         stream=None):
    """Token indices of the listed pools then each row's tail, and counts."""
    rows, pcap = int(pools.shape[0]), int(pools.shape[1])
    out = torch.empty((rows, out_cap), dtype=torch.int32, device=pools.device)
    cnt = torch.empty(rows, dtype=torch.int32, device=pools.device)
    st = load().indexer_expand_pools(_ptr(pools), pcap, _ptr(pool_counts), _ptr(row_lens), rows,
                                     pool_size, _ptr(out), out_cap, _ptr(cnt), _stream(stream))
    _check("indexer_expand_pools", st)
    return out, cnt


def indexer_decode_logits(q, weights, index_cache, block_table, row_seq_lens, next_n: int,
                          topk: int = MAX_TOPK, out_logits=None, workspace=None, dev_error=None,
                          stream=None):
    R = int(block_table.shape[0])
    rows = R * next_n
    ld = int(block_table.shape[1]) * PAGE_TOKENS
    if out_logits is None:
        out_logits = torch.full((rows, ld), float("nan"), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = decode_workspace(R, next_n, topk, q.device)
    st = load().indexer_decode_logits(
        _ptr(q), _ptr(weights), _ptr(index_cache), int(index_cache.shape[0]), _ptr(block_table),
        int(block_table.stride(0)), int(block_table.shape[1]), _ptr(row_seq_lens), R, next_n,
        int(q.shape[1]), int(q.shape[2]), topk, _ptr(out_logits), int(out_logits.stride(0)),
        _ptr(workspace), int(workspace.numel() * workspace.element_size()), _ptr(dev_error),
        _stream(stream))
    _check("indexer_decode_logits", st)
    return out_logits


def indexer_plan_prefill_chunks(seq_lens, query_lens, workspace_tokens: int,
                                logits_budget_bytes: int):
    import numpy as np
    sl, ql = _host_i32(seq_lens), _host_i32(query_lens)
    lib = load()
    cap = 64
    while True:
        buf = np.zeros((cap, 4), np.int32)
        n = C.c_int32(0)
        st = lib.indexer_plan_prefill_chunks(sl.ctypes.data, ql.ctypes.data, sl.shape[0],
                                             workspace_tokens, logits_budget_bytes,
                                             buf.ctypes.data, cap, C.byref(n))
        if st == 5:  # capacity
            cap = int(n.value)
            continue
        _check("indexer_plan_prefill_chunks", st)
        return [tuple(int(v) for v in buf[i]) for i in range(n.value)]


def indexer_prefill_workspace_bytes(seq_lens_host, query_lens_host, topk: int,
                                    workspace_tokens: int, logits_budget_bytes: int) -> int:
    sl, ql = _host_i32(seq_lens_host), _host_i32(query_lens_host)
    out = C.c_size_t(0)
    _check("indexer_prefill_workspace_bytes",
           load().indexer_prefill_workspace_bytes(sl.ctypes.data, ql.ctypes.data, sl.shape[0], topk,
                                                  workspace_tokens, logits_budget_bytes,
                                                  C.byref(out)))
    return int(out.value)


def indexer_prefill_topk(q, weights, index_cache, block_table, seq_lens, query_start_loc,
                         seq_lens_host, query_lens_host, topk: int = MAX_TOPK,
                         workspace_tokens: int = 40 * 8192, logits_budget_bytes: int = 512 << 20,
                         out_idx=None, workspace=None, dev_error=None, stream=None):
    sl, ql = _host_i32(seq_lens_host), _host_i32(query_lens_host)
    total_q = int(q.shape[0])
    if out_idx is None:
        out_idx = torch.empty((total_q, topk), dtype=torch.int32, device=q.device)
    if workspace is None:
        n = indexer_prefill_workspace_bytes(sl, ql, topk, workspace_tokens, logits_budget_bytes)
        workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=q.device)
    st = load().indexer_prefill_topk(
        _ptr(q), _ptr(weights), _ptr(index_cache), int(index_cache.shape[0]), _ptr(block_table),
        int(block_table.stride(0)), int(block_table.shape[1]), _ptr(seq_lens),
        _ptr(query_start_loc), sl.ctypes.data, ql.ctypes.data, sl.shape[0], int(q.shape[1]),
        int(q.shape[2]), topk, workspace_tokens, logits_budget_bytes, _ptr(out_idx),
        _ptr(workspace), int(workspace.numel() * workspace.element_size()), _ptr(dev_error),
        _stream(stream))
    _check("indexer_prefill_topk", st)
    return out_idx


def indexer_prefill_topk_values(q, weights, index_cache, block_table, seq_lens, query_start_loc,
                                seq_lens_host, query_lens_host, topk: int = MAX_TOPK,
                                compress_ratio: int = 1, dcp_rank: int = 0, dcp_world: int = 1,
                                dcp_interleave: int = 1, workspace_tokens: int = 40 * 8192,
                                logits_budget_bytes: int = 512 << 20, out_idx=None, out_val=None,
                                workspace=None, dev_error=None, stream=None):
    """Prefill top-k with the selected logits on one rank of a compressed and
    / or key-sharded cache. Returns (out_idx int32, out_val float32)."""
    sl, ql = _host_i32(seq_lens_host), _host_i32(query_lens_host)
    total_q = int(q.shape[0])
    if out_idx is None:
        out_idx = torch.empty((total_q, topk), dtype=torch.int32, device=q.device)
    if out_val is None:
        out_val = torch.empty((total_q, topk), dtype=torch.float32, device=q.device)
    if workspace is None:
        n = indexer_prefill_workspace_bytes(sl, ql, topk, workspace_tokens, logits_budget_bytes)
        workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=q.device)
    st = load().indexer_prefill_topk_values(
        _ptr(q), _ptr(weights), _ptr(index_cache), int(index_cache.shape[0]), _ptr(block_table),
        int(block_table.stride(0)), int(block_table.shape[1]), _ptr(seq_lens),
        _ptr(query_start_loc), sl.ctypes.data, ql.ctypes.data, sl.shape[0], int(q.shape[1]),
        int(q.shape[2]), topk, compress_ratio, dcp_rank, dcp_world, dcp_interleave,
        workspace_tokens, logits_budget_bytes, _ptr(out_idx), _ptr(out_val), _ptr(workspace),
        int(workspace.numel() * workspace.element_size()), _ptr(dev_error), _stream(stream))
    _check("indexer_prefill_topk_values", st)
    return out_idx, out_val


def indexer_profile_events(start_event=None, stop_event=None):
    """Records the given torch.cuda.Event pair around every score/select launch
    made from this thread (None, None turns it off)."""
    a = C.c_void_p(start_event.cuda_event) if start_event is not None else None
    b = C.c_void_p(stop_event.cuda_event) if stop_event is not None else None
    _check("indexer_profile_events", load().indexer_profile_events(a, b))


def indexer_trace_buffer(buffer=None):
    """Per-CTA trace stamps of later score/select launches go to ``buffer``
    (a uint64/int64 CUDA tensor of >= 128 * SM-count entries: 64 per tile
    stream, two streams per SM); None turns it off."""
    if buffer is None:
        _check("indexer_trace_buffer", load().indexer_trace_buffer(None, 0))
    else:
        _check("indexer_trace_buffer", load().indexer_trace_buffer(
            _ptr(buffer), int(buffer.numel() * buffer.element_size())))


def indexer_debug_decode_plan(num_reqs: int, next_n: int, topk: int = MAX_TOPK):
    """Where the decode work split lives in a workspace: returns (offsets
    dict of byte offsets, grid, (penalty, divisor))."""
    offs = (_I64 * 4)()
    grid = _I32(0)
    pen = (_I32 * 2)()
    _check("indexer_debug_decode_plan",
           load().indexer_debug_decode_plan(num_reqs, next_n, topk, offs, C.byref(grid), pen))
    names = ("wr_tile_start", "cta_tile", "row_ctas", "cta_row")
    return dict(zip(names, [int(v) for v in offs])), int(grid.value), (int(pen[0]), int(pen[1]))


def indexer_debug_divide(a, b, stream=None):
    """(the insert's quotient, the IEEE quotient) of float32 tensors a / b."""
    q = torch.empty_like(a)
    qi = torch.empty_like(a)
    st = load().indexer_debug_divide(_ptr(a), _ptr(b), int(a.numel()), _ptr(q), _ptr(qi),
                                     _stream(stream))
    _check("indexer_debug_divide", st)
    return q, qi


def indexer_debug_wait_limit(limit_ns: int = 0, stall_split_rows: bool = False):
    """Score/select launches from this thread give up their waits after
    ``limit_ns`` (0 restores the 2 s default); with ``stall_split_rows`` their
    split-row waits wait for a segment that never comes. For failure-detection
    tests."""
    _check("indexer_debug_wait_limit",
           load().indexer_debug_wait_limit(int(limit_ns), 1 if stall_split_rows else 0))


def indexer_decode_topk_noalloc(q, weights, index_cache, block_table, row_seq_lens, next_n: int,
                                topk: int = MAX_TOPK, out_idx=None, dev_error=None, stream=None):
    """indexer_decode_topk on the library's own scratch, for callers that
    cannot allocate a workspace (the output buffer is the caller's)."""
    R = int(block_table.shape[0])
    if out_idx is None:
        out_idx = torch.empty((R * next_n, topk), dtype=torch.int32, device=q.device)
    st = load().indexer_decode_topk_noalloc(
        _ptr(q), _ptr(weights), _ptr(index_cache), int(index_cache.shape[0]), _ptr(block_table),
        int(block_table.stride(0)), int(block_table.shape[1]), _ptr(row_seq_lens), R, next_n,
        int(q.shape[1]), int(q.shape[2]), topk, _ptr(out_idx), _ptr(dev_error), _stream(stream))
    _check("indexer_decode_topk_noalloc", st)
    return out_idx


# ---------------------------------------------------------------------------
# attention over a paged key/value cache, and the pages of the caches
#
# These calls look at their tensors' device, type, shape and strides and raise
# IndexerError (invalid argument or unsupported) before anything is enqueued.
# What they allocate (outputs, workspaces) belongs to the stream they run on.
# ---------------------------------------------------------------------------

_INVALID = 1
_I32T = torch.int32


def _refuse(name, what, status=_INVALID):
    raise IndexerError(name, status, what)


def _need_i32(name, what, t, *shape):
    """An int32 tensor of that shape (None: any size), contiguous in its last dimension."""
    if not isinstance(t, torch.Tensor) or t.dtype is not _I32T:
        _refuse(name, f"{what} must be an int32 tensor")
    got = t.shape
    if got != shape:
        if len(got) != len(shape):
            _refuse(name, f"{what} has shape {tuple(got)}")
        for a, n in zip(got, shape):
            if n is not None and a != n:
                _refuse(name, f"{what} has shape {tuple(got)}")
    if not t.is_contiguous() and t.stride(-1) != 1 and got[-1] > 1:
        _refuse(name, f"{what} must be contiguous in its last dimension")


def _need_table(name, block_table, rows=None):
    """(width, row stride) of a block table."""
    _need_i32(name, "block_table", block_table, rows, None)
    n, width = block_table.shape
    if width < 1:
        _refuse(name, "block_table has no columns")
    stride = block_table.stride(0)
    if stride < width:
        if n > 1:
            _refuse(name, "block_table's rows overlap")
        stride = width
    return width, stride


def _need_error(name, dev_error):
    if dev_error is not None and not (isinstance(dev_error, torch.Tensor)
                                      and dev_error.element_size() == 4 and dev_error.numel() >= 1):
        _refuse(name, "dev_error must be a tensor of a 32-bit word")


def _need_device(name, first, *others):
    """The index of the CUDA device that all the tensors are on."""
    if not first.is_cuda:
        _refuse(name, "tensors must be on a CUDA device")
    index = first.get_device()
    for t in others:
        if t is not None and t.get_device() != index:
            _refuse(name, "tensors are on different devices")
    return index


class _On:
    """Allocates on, and hands out, the stream a call runs on: the current one
    of the tensors' device, or the caller's."""

    __slots__ = ("guard", "index")

    def __init__(self, index, stream):
        self.guard = None
        self.index = index
        if stream is None and torch._C._cuda_getDevice() == index:
            return
        device = torch.device("cuda", index)
        if stream is None:
            stream = torch.cuda.current_stream(device)
        elif isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=device)
        self.guard = torch.cuda.stream(stream)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        # (the handle that current_stream().cuda_stream gives, without the stream object)
        return torch._C._cuda_getCurrentRawStream(self.index)

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


@functools.lru_cache(maxsize=256)
def _attend_workspace_bytes(device, *sizes):
    n = C.c_size_t(0)
    _check("indexer_attend_workspace_bytes", load().indexer_attend_workspace_bytes(*sizes, C.byref(n)))
    return n.value


def attend_workspace(num_tokens: int, num_reqs: int, num_heads: int, num_kv_heads: int,
                     head_dim: int, device="cuda"):
    """Workspace for indexer_attend_paged / indexer_attend_selected / indexer_attend_tree calls on that
    device, none of whose sizes is larger than these."""
    with torch.cuda.device(device):
        n = _attend_workspace_bytes(torch.cuda.current_device(), num_tokens, num_reqs, num_heads,
                                    num_kv_heads, head_dim)
    return torch.empty(n, dtype=torch.uint8, device=device)


def indexer_attend_paged(q, k_cache, v_cache, block_table, seq_lens, query_start_loc,
                         max_query_len: int = 0, scale=None, window: int = 0, sinks: int = 0,
                         out=None, lse=None, workspace=None, dev_error=None, stream=None):
    """Causal attention of every request's new tokens over its paged cache:
    q [tokens, heads, dim] (bf16 or fp16, dim 64 or 128), k_cache and v_cache
    [pages, 64, kv heads, dim] of the same type (any strides that keep dim
    contiguous), block_table int32 [requests, width], seq_lens int32 [requests]
    (keys, the new ones among them), query_start_loc int32 [requests + 1].
    window > 0: a token sees the last `window` keys up to its own, and the
    first `sinks` keys. max_query_len (new tokens of the longest request) is a
    hint that chooses the kernel, for small and windowed steps the faster one;
    0 and anything above the tokens count as all of them. scale defaults to
    dim ** -0.5. Returns (out like q, lse float32 [tokens, heads])."""
    return _native().attend(0, q, k_cache, v_cache, block_table, query_start_loc, seq_lens, None, scale, out, lse,
                            workspace, dev_error, stream, max_query_len, window, sinks, None, None)


def indexer_attend_selected(q, k_cache, v_cache, block_table, indices, query_start_loc, scale=None,
                            out=None, lse=None, workspace=None, dev_error=None, stream=None):
    """Attention of every token to the keys listed for it: indices int32
    [tokens, topk], positions of the token's request, entries < 0 empty (the
    output of indexer_decode_topk / indexer_prefill_topk). Other arguments and
    the result as indexer_attend_paged."""
    return _native().attend(1, q, k_cache, v_cache, block_table, query_start_loc, None, indices, scale, out, lse,
                            workspace, dev_error, stream, 0, 0, 0, None, None)


def indexer_attend_tree(q, k_cache, v_cache, block_table, seq_lens, query_start_loc, masks,
                        max_query_len: int = 0, positions=None, scale=None, window: int = 0,
                        sinks: int = 0, out=None, lse=None, workspace=None, dev_error=None,
                        stream=None):
    """Attention of trees of drafted tokens over the paged cache: a request's new
    tokens see every key before them (with a window: those that the token's
    position, int32 [tokens], leaves) and the new tokens that their rows of masks
    (int32 [tokens, words], bit j: the request's new token j) name. masks and
    positions are what indexer_plan_tree makes. Other arguments and the result as
    indexer_attend_paged; max_query_len (nodes of the largest tree) is a hint."""
    return _native().attend(2, q, k_cache, v_cache, block_table, query_start_loc, seq_lens, None, scale, out, lse,
                            workspace, dev_error, stream, max_query_len, window, sinks, masks, positions)


def _pools(name, pools, num_pages):
    """The pools as idx_page_pool entries: tensors of [pages, ...] whose pages are contiguous."""
    out = (PagePool * max(1, len(pools)))()
    for i, t in enumerate(pools):
        if not isinstance(t, torch.Tensor) or t.dim() < 2:
            _refuse(name, "a pool must be a tensor [pages, ...]")
        pages = t.shape[0]
        if pages < 1 or (num_pages is not None and pages != num_pages):
            _refuse(name, "the pools differ in pages")
        num_pages = pages
        size = t.element_size()
        if t.is_contiguous():
            n = stride = t.numel() // pages * size
        else:
            one = t[0]
            n = one.numel() * size
            stride = t.stride(0) * size if pages > 1 else n
            if not one.is_contiguous():
                _refuse(name, "a pool's pages must be contiguous")
        at = t.data_ptr()
        if n % 16 or at % 16:
            _refuse(name, "a pool's pages must be multiples of 16 bytes")
        p = out[i]
        p.base, p.page_stride, p.page_bytes = at, stride, n
    return out, num_pages


def _ok(name, st):
    if st:
        _check(name, st)


def _at(t):
    return None if t is None else t.data_ptr()


def _need_rows(name, block_table, seq_lens, ref_counts):
    width, stride = _need_table(name, block_table)
    _need_i32(name, "seq_lens", seq_lens, block_table.shape[0])
    _need_i32(name, "ref_counts", ref_counts, None)
    return block_table.shape[0], width, stride


def indexer_copy_pages(pools, src, dst, dev_error=None, stream=None):
    """Page src[i] to page dst[i] (int32 [n]) in every pool (tensors [pages, ...]); negative
    entries are skipped."""
    name = "indexer_copy_pages"
    if not pools:
        _refuse(name, "no pools")
    _need_i32(name, "src", src, None)
    _need_i32(name, "dst", dst, src.shape[0])
    _need_error(name, dev_error)
    arr, pages = _pools(name, pools, None)
    index = _need_device(name, src, dst, dev_error, *pools)
    with _On(index, stream) as s:
        _ok(name, load().indexer_copy_pages(arr, len(pools), pages, _at(src), _at(dst),
                                               src.shape[0], _at(dev_error), s))


def indexer_fork_pages(pools, block_table, seq_lens, ref_counts, parents, children, copy_src=None,
                       copy_dst=None, dev_error=None, stream=None):
    """Makes block-table row children[i] (empty before) a copy of row parents[i]: full pages
    shared, a partial last page copied to the lowest free page in every pool. block_table,
    seq_lens, ref_counts (int32) and the pools change in place. Returns (copy_src, copy_dst)
    int32 [n]: the page copies made, then -1."""
    name = "indexer_fork_pages"
    rows_n, width, bt_stride = _need_rows(name, block_table, seq_lens, ref_counts)
    _need_i32(name, "parents", parents, None)
    n = parents.shape[0]
    _need_i32(name, "children", children, n)
    for what, t in (("copy_src", copy_src), ("copy_dst", copy_dst)):
        if t is not None:
            _need_i32(name, what, t, n)
    _need_error(name, dev_error)
    arr, pages = _pools(name, pools, ref_counts.shape[0])
    index = _need_device(name, block_table, seq_lens, ref_counts, parents, children, copy_src, copy_dst,
                         dev_error, *pools)
    with _On(index, stream) as s:
        if copy_src is None:
            copy_src = torch.empty_like(parents)
        if copy_dst is None:
            copy_dst = torch.empty_like(parents)
        _ok(name, load().indexer_fork_pages(
            arr, len(pools), pages, _at(block_table), bt_stride, width, rows_n,
            _at(seq_lens), _at(ref_counts), _at(parents), _at(children), n, _at(copy_src), _at(copy_dst), _at(dev_error), s))
    return copy_src, copy_dst


def indexer_free_pages(block_table, seq_lens, ref_counts, rows, dev_error=None, stream=None):
    """Frees the block-table rows listed in rows (int32, distinct): their pages lose a reference
    in ref_counts, their seq_lens become 0, in place."""
    name = "indexer_free_pages"
    rows_n, width, bt_stride = _need_rows(name, block_table, seq_lens, ref_counts)
    _need_i32(name, "rows", rows, None)
    _need_error(name, dev_error)
    index = _need_device(name, block_table, seq_lens, ref_counts, rows, dev_error)
    with _On(index, stream) as s:
        _ok(name, load().indexer_free_pages(
            _at(block_table), bt_stride, width, rows_n,
            _at(seq_lens), _at(ref_counts), ref_counts.shape[0], _at(rows),
            rows.shape[0], _at(dev_error), s))


@functools.lru_cache(maxsize=256)
def _compact_workspace_bytes(pages):
    n = C.c_size_t(0)
    _check("indexer_compact_workspace_bytes",
           load().indexer_compact_workspace_bytes(pages, C.byref(n)))
    return n.value


def indexer_compact_pages(pools, block_table, seq_lens, ref_counts, remap=None, num_live=None,
                          workspace=None, dev_error=None, stream=None):
    """Moves the pages in use to the front of the pools (data, ref_counts and block_table in
    place). Returns (remap int32 [pages]: a page's new number, -1 if it was free; num_live int32
    [1] on the device: pages in use)."""
    name = "indexer_compact_pages"
    rows_n, width, bt_stride = _need_rows(name, block_table, seq_lens, ref_counts)
    pages = ref_counts.shape[0]
    if remap is not None:
        _need_i32(name, "remap", remap, pages)
    if num_live is not None:
        _need_i32(name, "num_live", num_live, 1)
    _need_error(name, dev_error)
    arr, pages = _pools(name, pools, pages)
    index = _need_device(name, block_table, seq_lens, ref_counts, remap, num_live, workspace, dev_error, *pools)
    lib = load()
    with _On(index, stream) as s:
        if remap is None:
            remap = torch.empty(pages, dtype=torch.int32, device=ref_counts.device)
        if num_live is None:
            num_live = torch.empty(1, dtype=torch.int32, device=ref_counts.device)
        if workspace is None:
            workspace = torch.empty(_compact_workspace_bytes(pages), dtype=torch.uint8,
                                    device=ref_counts.device)
        _ok(name, lib.indexer_compact_pages(
            arr, len(pools), pages, _at(block_table), bt_stride, width, rows_n,
            _at(seq_lens), _at(ref_counts), _at(remap), _at(num_live), _at(workspace), workspace.numel() * workspace.element_size(),
            _at(dev_error), s))
    return remap, num_live


# ---------------------------------------------------------------------------
# new and drafted tokens in the caches
# ---------------------------------------------------------------------------


def indexer_append_kv(k, v, k_cache, v_cache, slot_mapping, q=None, positions=None, rotary=None,
                      interleaved: bool = False, q_out=None, dev_error=None, stream=None):
    """Writes new tokens' keys and values k, v [tokens, kv heads, dim] (bf16 or
    fp16, dim 64 or 128) to their slots (slot_mapping int64 [tokens]: page * 64 +
    token, negative: padding) of k_cache, v_cache [pages, 64, kv heads, dim], in
    place. With rotary (float32 [positions, rotary_dim]: cosines, then sines; rotary_dim
    a multiple of 16) the first rotary_dim values of the keys, and of the
    queries q [tokens, heads, dim] if given, are rotated to their positions (int32
    [tokens]) on the way: value i with i + rotary_dim / 2, or neighbours when
    interleaved. Any strides that keep dim contiguous and are multiples of 8. Returns
    the rotated queries (q_out; q itself may be given), None without q."""
    return _native().append_kv(k, v, k_cache, v_cache, slot_mapping, q, positions, rotary, interleaved, q_out,
                               dev_error, stream)


def indexer_insert_keys_mxfp4(k, slot_mapping, index_cache, values=None, dev_error=None, stream=None):
    """Quantises k (bf16 [T, 128], rows of any stride that is a multiple of 8) to MXFP4 entries and
    writes them into the paged index cache (uint8 [pages, 4352]) at slot_mapping (int64 [T]); in
    place. values (bf16 [T, 128], contiguous) gets what the entries stand for."""
    return _native().insert_keys_mxfp4(k, slot_mapping, index_cache, values, dev_error, stream)


def indexer_plan_tree(parents, seq_lens, query_start_loc, max_query_len: int, window: int = 0,
                      sinks: int = 0, max_path: int = 0, masks=None, positions=None, paths=None,
                      dev_error=None, stream=None):
    """What trees of drafted tokens ask of attention, from their nodes' parents (int32 [tokens],
    indices among the request's new tokens, -1 for a root). Returns (masks int32 [tokens, words]:
    every node and its ancestors, with a window those that it leaves; positions int32 [tokens]; paths
    int32 [tokens, max_path]: the places of a node and its ancestors in the cache, -1 after, None
    with max_path 0). max_query_len: nodes of the largest tree (words = ceil(max_query_len / 32))."""
    return _native().plan_tree(parents, seq_lens, query_start_loc, max_query_len, window, sinks, max_path, masks,
                               positions, paths, dev_error, stream)


def indexer_commit_tree(pools, block_table, seq_lens, query_start_loc, accepted, ref_counts=None,
                        dev_error=None, stream=None):
    """Keeps every request's accepted nodes (accepted int32 [requests, n]: ascending, then -1) of its
    tree of new tokens and drops the others: in every pool (tensors [pages, 64, ...] of keys or
    values, uint8 index caches [pages, 8448] or [pages, 4352], none twice) their tokens move to the
    tree's first places, seq_lens becomes L - Q + accepted nodes, and the pages that a row no longer
    holds lose a reference in ref_counts (int32 [pages]), all in place. Rows of block_table are the
    requests."""
    _native().commit_tree(pools, block_table, seq_lens, query_start_loc, accepted, ref_counts, dev_error, stream)
