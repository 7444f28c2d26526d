"""fp16 attention where one key outweighs all others together and they still hold a share of the
output: a long tail of weights near 2^-25 of the largest, which fp16 has no values for beside 1.

Weights are held in fp16 as multiples of 2^15 (row-block and list kernels) or of at least 2^7 (chunk
kernel) of the largest one, so that one below fp16's normal range is off by 2^-25 of those: n 2^-40
or n 2^-32 of max |v| in all, where the tolerance of test_gpu_attend has n 2^-25. The outputs are
kept in fp16's normal range by values of some thousand.
"""
import math

import pytest
import torch

from test_gpu_attend import DEV, FP, PAGE, Batch, _lib  # noqa: F401

pytestmark = pytest.mark.gpu

GAP = 17.5   # e^-17.5 = 2^-25.2


def _batch(ql, kl, heads, kv, dim, seed, top):
    """Every query scores key top[b] of its request GAP above the others, which lie near 0; values
    of 0 there, of 2000 on average elsewhere."""
    b = Batch(ql, kl, heads, kv, dim, FP, seed=seed)
    b.q.zero_()
    b.q[:, :, 0] = math.sqrt(dim)
    for r, n in enumerate(kl):
        for i in range(-(-n // PAGE)):
            m = min(PAGE, n - i * PAGE)
            page = int(b.table[r, i])
            b.k[page, :m] = 0
            b.k[page, :m, :, 0] = 0.1 * torch.randn((m, kv), generator=b.gen, device=DEV).to(FP)
            b.v[page, :m] = (2000 + 100 * torch.randn((m, kv, dim), generator=b.gen, device=DEV)).to(FP)
        page, slot = int(b.table[r, top[r] // PAGE]), top[r] % PAGE
        b.k[page, slot, :, 0] = GAP
        b.v[page, slot] = 0
    return b


def _want(b, terms, fine, **kw):
    """The reference with its tolerance's terms * 2^-25 max |v| made terms * 2^-fine."""
    out, lse, tol, ltol = b.reference(**kw)
    most = torch.cat([b.keys(r)[1].abs().amax((0, 2)).repeat_interleave(b.heads // b.kv_heads).expand(q, -1)
                      for r, q in enumerate(b.ql)])
    return out, lse, tol - (terms[:, None] * (2.0 ** -25 - 2.0 ** -fine) * most)[:, :, None], ltol


def _positions(b):
    return torch.cat([torch.arange(n - q, n, device=DEV) for q, n in zip(b.ql, b.kl)]).double()


# single tokens and rows that share a block (clusters, then units cut by a plan), chunks (planned by
# their own blocks, then by a kernel): new tokens, keys, heads, kv heads, bits
CASES = [([1, 2], [1000, 4000], 8, 2, 40), ([1], [65536], 4, 1, 40), ([1] * 40, [3000] * 40, 16, 4, 40),
         ([40], [4000], 8, 2, 32), ([300, 30], [30000, 65536], 8, 2, 32)]


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("where", ["first", "middle", "late"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_tail_of_a_paged_row(case, where, dim):
    ql, kl, heads, kv, fine = CASES[case]
    top = [{"first": 0, "middle": n // 2, "late": n - q}[where] for q, n in zip(ql, kl)]
    b = _batch(ql, kl, heads, kv, dim, 500 + case, top)
    b.check(b.attend(), _want(b, _positions(b) + 1, fine))


# clusters, CTAs and warps per list
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("tokens,heads,kv,topk", [(2, 8, 2, 512), (60, 16, 8, 2048), (900, 8, 2, 100), (200, 40, 1, 700)])
def test_tail_of_a_list(tokens, heads, kv, topk, dim):
    b = _batch([tokens], [4000], heads, kv, dim, 520, [5])
    idx = torch.stack([torch.randperm(3000, generator=b.gen, device=DEV)[:topk] for _ in range(tokens)])
    idx = torch.where((idx == 5).any(1)[:, None], idx, torch.cat([torch.full_like(idx[:, :1], 5), idx[:, 1:]], 1))
    idx = idx.to(torch.int32)
    terms = torch.full((tokens,), float(topk), dtype=torch.float64, device=DEV)
    b.check(b.attend_selected(idx), _want(b, terms, 40, indices=idx))


def test_weights_stay_in_range_as_the_maximum_climbs():
    """Scores that climb by less than the chunk kernel's lazy step from tile to tile, with values near
    fp16's largest: weights reach 2^15 of their reference and no product leaves fp32."""
    for dim in (64, 128):
        b = Batch([200, 1], [2000, 300], 8, 2, dim, FP, seed=540)
        b.q.zero_()
        b.q[:, :, 0] = math.sqrt(dim)
        for r, n in enumerate(b.kl):
            for i in range(-(-n // PAGE)):
                m = min(PAGE, n - i * PAGE)
                page = int(b.table[r, i])
                b.k[page, :m] = 0
                # 5.3 nats (7.6 in log 2) a tile of 128 keys
                climb = 5.3 * (torch.arange(i * PAGE, i * PAGE + m, device=DEV) // 128)
                b.k[page, :m, :, 0] = climb[:, None].to(FP)
                b.v[page, :m] = 60000.0 * torch.sign(torch.randn((m, 2, dim), generator=b.gen, device=DEV)).to(FP)
        b.check(b.attend(), b.reference())
