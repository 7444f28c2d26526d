"""Trees on the GPU at the sizes where their kernels change: paths too wide to be written together, and batches whose
plan does not fit in shared memory."""
import random

import pytest
import torch

import sparse_attention_indexer_block_gb300 as saib
from test_gpu_attend import BF, DEV, FP, _lib  # noqa: F401
from test_gpu_tree import TreeBatch, _i32, _plan, _trees

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("width", [1, 2, 31, 1023, 1024, 1025, 1300])
def test_plan_paths_of_any_width(width):
    trees = [[-1] + list(range(1199)), _trees([40], 1)[0], [-1] * 33, [-1] + list(range(32))]
    kl = [1300, 40, 9000, 34]
    start = [0]
    for t in trees:
        start.append(start[-1] + len(t))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    masks, positions, paths = saib.indexer_plan_tree(_i32([p for t in trees for p in t]), _i32(kl), _i32(start), 1200,
                                                     max_path=width, dev_error=err)
    torch.cuda.synchronize()
    assert int(err) == (8 if width < 1200 else 0)
    want = _plan(trees, kl, -(-1200 // 32), width)
    assert masks.tolist() == want[0] and positions.tolist() == want[1] and paths.tolist() == want[2]


@pytest.mark.parametrize("dim,dtype", [(64, FP), (64, BF), (128, BF)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 3)])
def test_tree_of_more_requests_than_a_plan_holds(dim, dtype, window, sinks):
    """Units of one and of two slots, planned from memory."""
    rng = random.Random(6)
    ql = [rng.choice([0, 1, 2, 9, 9, 20, 40]) for _ in range(1100)]
    kl = [q + rng.randrange(0, 200) for q in ql]
    b = TreeBatch(ql, kl, 8, 1, dim, dtype, seed=50)
    b.check(b.attend_tree(window=window, sinks=sinks), b.reference_tree(window, sinks))
