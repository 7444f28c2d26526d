"""Trees on the GPU: a row that computes with a NaN shows it in out and lse, whichever kernel runs it and however its
keys are cut over the CTAs, and no other row changes."""
import pytest
import torch

from test_gpu_attend import BF, DEV, FP, PAGE, _lib  # noqa: F401
from test_gpu_tree import TreeBatch

pytestmark = pytest.mark.gpu

# (new tokens, keys, heads, kv heads): units cut over several CTAs, few and many; whole units; clusters; blocks of rows
CUT = [([60, 8], [20000, 20000], 8, 1), ([30] * 20, [3000] * 20, 16, 2), ([95], [8000], 32, 8)]
OTHERS = [([60, 140], [260, 400], 8, 2), ([8], [1000], 32, 8), ([4], [4500], 32, 8), ([2] * 200, [300] * 200, 8, 4)]


def _same(got, want, rows):
    for g, w in zip(got, want):
        assert torch.equal(g[rows], w[rows])


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("ql,kl,heads,kv", CUT + OTHERS)
def test_rows_of_nan_queries_are_nan(ql, kl, heads, kv, dtype, dim):
    b = TreeBatch(ql, kl, heads, kv, dim, dtype, seed=3, tree_seed=2)
    clean = b.attend_tree()
    nan = torch.zeros((b.rows, heads), dtype=torch.bool, device=DEV)
    nan[0, 0] = nan[b.rows // 2] = nan[b.rows - 1, heads - 1] = True
    b.q = torch.where(nan[..., None], float("nan"), b.q)
    got = b.attend_tree()
    assert got[0][nan].isnan().all() and got[1][nan].isnan().all()
    _same(got, clean, ~nan)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("ql,kl,heads,kv", CUT)
def test_rows_over_pages_of_nan_keys_are_nan(ql, kl, heads, kv, dtype, dim):
    """Whole pieces of NaN scores before, between and behind pieces of finite ones."""
    b = TreeBatch(ql, kl, heads, kv, dim, dtype, seed=4, tree_seed=2)
    clean = b.attend_tree()
    full, n = kl[0] // PAGE, b.start_h[1]
    for first, last in ((0, full // 3), (full // 3, 2 * full // 3), (2 * full // 3, full - 2)):
        pages = b.table[0, first:last].long()
        keep = b.k[pages].clone()
        b.k[pages] = float("nan")
        got = b.attend_tree()
        b.k[pages] = keep
        assert got[0][:n].isnan().all() and got[1][:n].isnan().all()
        _same(got, clean, slice(n, None))
