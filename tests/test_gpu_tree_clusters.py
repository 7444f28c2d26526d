"""The clusters that trees run in, read from captured calls: eight blocks, and sixteen where units are few and long
and the device has room for them."""
import ctypes as C

import pytest
import torch

import sparse_attention_indexer_block_gb300 as saib
from test_gpu_attend import BF, DEV, FP, _lib  # noqa: F401
from test_gpu_tree import TreeBatch

pytestmark = pytest.mark.gpu


class KernelNode(C.Structure):
    """CUDA_KERNEL_NODE_PARAMS of the driver API."""
    _fields_ = [("func", C.c_void_p), ("grid", C.c_uint * 3), ("block", C.c_uint * 3), ("shared", C.c_uint),
                ("params", C.c_void_p), ("extra", C.c_void_p), ("kern", C.c_void_p), ("ctx", C.c_void_p)]


def _kernels(call):
    """(blocks, blocks of a cluster) of every kernel that a captured call launches."""
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    cuda, raw = C.CDLL("libcuda.so.1"), C.c_void_p(graph.raw_cuda_graph())
    n = C.c_size_t(0)
    assert cuda.cuGraphGetNodes(raw, None, C.byref(n)) == 0
    nodes = (C.c_void_p * n.value)()
    assert cuda.cuGraphGetNodes(raw, nodes, C.byref(n)) == 0
    out = []
    for node in nodes:
        kind = C.c_int(-1)
        assert cuda.cuGraphNodeGetType(C.c_void_p(node), C.byref(kind)) == 0
        if kind.value != 0:
            continue
        k, value = KernelNode(), (C.c_uint * 16)()
        assert cuda.cuGraphKernelNodeGetParams_v2(C.c_void_p(node), C.byref(k)) == 0
        assert cuda.cuGraphKernelNodeGetAttribute(C.c_void_p(node), 4, C.byref(value)) == 0   # cluster dimension
        out.append((k.grid[0], max(1, value[0])))
    return out


def _width(units, tiles):
    """The rule: eight blocks, sixteen for few units of many tiles, halved until they fit the device (two a SM) and have
    a tile for every two of them."""
    c = 16 if units <= 8 and tiles > 32 else 8
    while c > 1 and (units * c > 2 * torch.cuda.get_device_properties(DEV).multi_processor_count or c >= 2 * tiles):
        c //= 2
    return c


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("ql,kl,heads,kv,dim,units,wide", [
    ([4], [4500], 32, 8, 128, 8, 16), ([4, 8], [9000, 5000], 8, 2, 128, 8, 16), ([16], [12000], 8, 1, 64, 8, 16),
    ([1], [7000], 16, 4, 64, 4, 16), ([1], [9], 16, 4, 64, 4, 2), ([8], [4500], 32, 8, 128, 16, 8),
    ([4], [1000], 32, 8, 128, 8, 8)])
def test_blocks_of_a_cluster(ql, kl, heads, kv, dim, units, wide, dtype):
    b = TreeBatch(ql, kl, heads, kv, dim, dtype, seed=40)
    assert _width(units, -(-b.width * 64 // (64 if dim == 128 else 128))) == wide
    got = b.attend_tree()
    ws = saib.attend_workspace(b.rows, len(ql), heads, kv, dim)
    out, lse = torch.empty_like(got[0]), torch.empty_like(got[1])

    def call():
        saib.indexer_attend_tree(b.q, b.k, b.v, b.table, b.lens, b.start, b.masks, max(ql), out=out, lse=lse, workspace=ws)

    assert _kernels(call) == [(units * wide, wide)]
    b.check(got, b.reference_tree())


def test_a_first_call_of_sixteen_may_be_captured():
    """What the choice asks of the device it may ask inside a capture."""
    import os
    import subprocess
    import sys
    code = """
import sys, torch
sys.path.insert(0, "tests")
import sparse_attention_indexer_block_gb300 as saib
from test_gpu_tree import TreeBatch, BF, DEV
saib.load()
b = TreeBatch([4], [4500], 32, 8, 128, BF, seed=41)
out, lse = torch.empty_like(b.q), torch.empty((4, 32), device=DEV)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    saib.indexer_attend_tree(b.q, b.k, b.v, b.table, b.lens, b.start, b.masks, 4, out=out, lse=lse)
graph.replay()
torch.cuda.synchronize()
want = b.attend_tree()
assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", code], check=True, cwd=root, timeout=300)
