"""Paged and selected-token attention on the GPU against the formula in 64 bits.

Tolerance of an output element (u = half a step of the type, eps / 2): the
weights p are rounded to the type before the second product and the output once
more, so u * (A + |out|) with A = sum p |v| / sum p; the scores and sums are
fp32: a score is off by at most (D + 2) 2^-24 X with X the row's largest scale *
sum |q k|, which moves a weight by that much relative, and a sum of n terms by n
2^-23 relative. fp16 weights below 2^-14 are off by 2^-25 of the largest weight
instead: n 2^-25 max |v| more. lse is off by the score's error, the sum's n
2^-23, and 2^-22 of its own size from the exponentials and the logarithm.
"""
import math

import pytest
import torch

import sparse_attention_indexer_block_gb300 as saib

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
PAGE = 64


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from sparse_attention_indexer_block_gb300 import build as libbuild
    libbuild.build()
    saib.load()
    torch.cuda.set_device(DEV)


class Batch:
    """Requests of ql new tokens over kl keys, their pages scattered over the pool; what lies
    past a length (slots of its last page, unused pages and table entries) is NaN or invalid."""

    def __init__(self, ql, kl, heads, kv_heads, dim, dtype, seed=0, extra_pages=3, layout="pages", q_pad=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.ql, self.kl, self.heads, self.kv_heads, self.dim, self.dtype = ql, kl, heads, kv_heads, dim, dtype
        pages = [-(-n // PAGE) for n in kl]
        total = sum(pages) + extra_pages
        order = torch.randperm(total, generator=g, device=DEV).tolist()
        self.width = max(1, max(pages)) + 2
        table = torch.full((len(kl), self.width), -7, dtype=torch.int32)
        shape = (total, PAGE, kv_heads, dim)
        k = torch.full(shape, float("nan"), device=DEV, dtype=dtype)
        v = torch.full(shape, float("nan"), device=DEV, dtype=dtype)
        at = 0
        for b, n in enumerate(pages):
            ids = order[at:at + n]
            at += n
            table[b, :n] = torch.tensor(ids, dtype=torch.int32)
            for i, page in enumerate(ids):
                m = min(PAGE, kl[b] - i * PAGE)
                for c in (k, v):
                    c[page, :m] = torch.randn((m, kv_heads, dim), generator=g, device=DEV).to(dtype)
        if layout == "heads":      # [pages, kv heads, 64, dim] in memory
            k, v = (c.transpose(1, 2).contiguous().transpose(1, 2) for c in (k, v))
        elif layout == "joint":    # K and V side by side in one array
            both = torch.stack([k, v], dim=1)
            k, v = both[:, 0], both[:, 1]
        self.k, self.v, self.table = k, v, table.to(DEV)
        start = [0]
        for q in ql:
            start.append(start[-1] + q)
        self.start_h, self.rows = start, start[-1]
        self.start = torch.tensor(start, dtype=torch.int32, device=DEV)
        self.lens = torch.tensor(kl, dtype=torch.int32, device=DEV)
        q = torch.randn((self.rows, heads, dim + q_pad), generator=g, device=DEV).to(dtype)
        self.q = q[:, :, :dim]
        self.gen = g

    def keys(self, b):
        n = self.kl[b]
        at = self.table[b, :-(-n // PAGE)].long()
        return (self.k[at].reshape(-1, self.kv_heads, self.dim)[:n].double(),
                self.v[at].reshape(-1, self.kv_heads, self.dim)[:n].double())

    def reference(self, window=0, sinks=0, indices=None, scale=None):
        """(out, lse, tolerance of out, tolerance of lse), 64-bit, row by row of the definition."""
        d, u = self.dim, torch.finfo(self.dtype).eps / 2
        scale = d ** -0.5 if scale is None else scale
        group = self.heads // self.kv_heads
        out = torch.zeros((self.rows, self.heads, d), dtype=torch.float64, device=DEV)
        lse = torch.full((self.rows, self.heads), -math.inf, dtype=torch.float64, device=DEV)
        tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
        for b, (nq, n) in enumerate(zip(self.ql, self.kl)):
            if n == 0 or nq == 0:
                continue
            k, v = self.keys(b)
            r0 = self.start_h[b]
            q = self.q[r0:r0 + nq].double()
            pos = torch.arange(nq, device=DEV) + (n - nq)
            key = torch.arange(n, device=DEV)
            if indices is None:
                see = key[None] <= pos[:, None]
                if window > 0:
                    see &= (pos[:, None] - key[None] < window) | (key[None] < sinks)
                times = see.double()
            else:
                idx = indices[r0:r0 + nq].long()
                times = torch.zeros((nq, n + 1), dtype=torch.float64, device=DEV)
                times.scatter_add_(1, torch.where(idx < 0, n, idx), torch.ones_like(idx, dtype=torch.float64))
                times = times[:, :n]
                see = times > 0
            for h in range(self.heads):
                kk, vv = k[:, h // group], v[:, h // group]
                x = torch.where(see, (q[:, h] @ kk.T) * scale + times.log(), -math.inf)
                size = torch.where(see, (q[:, h].abs() @ kk.abs().T) * scale, 0.0).amax(1)
                z = torch.logsumexp(x, 1)
                p = torch.exp(x - torch.where(z == -math.inf, 0.0, z)[:, None])
                o, a = p @ vv, p @ vv.abs()
                terms = see.sum(1).double()
                off = (d + 2) * 2.0 ** -24 * size + terms * 2.0 ** -23
                out[r0:r0 + nq, h], lse[r0:r0 + nq, h] = o, z
                t = u * (a + o.abs()) + 2 * off[:, None] * a
                if self.dtype == torch.float16:
                    t = t + (terms * 2.0 ** -25)[:, None] * vv.abs().amax()
                tol[r0:r0 + nq, h] = t
                ltol[r0:r0 + nq, h] = off + 2.0 ** -22 * (1 + z.abs().clamp(max=1e30))
        return out, lse, tol, ltol

    def check(self, got, want):
        (out, lse), (ro, rl, tol, ltol) = got, want
        empty = rl == -math.inf
        assert torch.equal(lse == -math.inf, empty)
        assert not out[empty].any() and torch.isfinite(out).all()
        bad = (out.double() - ro).abs() > tol
        assert not bad.any(), f"{int(bad.sum())} elements, first {bad.nonzero()[0].tolist()}: " \
            f"worst {((out.double() - ro).abs() / tol.clamp(min=1e-30)).max().item():.2f} of the tolerance"
        far = ((lse.double() - rl).abs() > ltol) & ~empty
        assert not far.any(), f"lse of {int(far.sum())} rows"

    def attend(self, **kw):
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        r = saib.indexer_attend_paged(self.q, self.k, self.v, self.table, self.lens, self.start,
                                      kw.pop("max_query_len", max(self.ql)), dev_error=err, **kw)
        torch.cuda.synchronize()
        assert int(err.item()) == 0, f"device error word {int(err.item())}"
        return r

    def attend_selected(self, indices, **kw):
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        r = saib.indexer_attend_selected(self.q, self.k, self.v, self.table, indices, self.start,
                                         dev_error=err, **kw)
        torch.cuda.synchronize()
        assert int(err.item()) == 0, f"device error word {int(err.item())}"
        return r


BF, FP = torch.bfloat16, torch.float16

# new tokens, keys, heads, kv heads
SHAPES = [
    ([1], [1], 1, 1),
    ([1], [1000], 32, 8),
    ([1] * 7, [64, 1, 63, 65, 128, 200, 0], 8, 1),
    ([2] * 5, [2, 3, 64, 66, 400], 16, 2),
    ([1, 5, 17, 3], [700, 5, 200, 64], 10, 2),           # a group of 5
    ([3, 1, 0, 2], [1, 0, 50, 2], 6, 2),                 # fewer keys than tokens, none, no tokens
    ([130, 1, 64], [130, 513, 300], 12, 4),              # a group of 3
    ([33, 7], [1100, 100], 48, 3),                       # a group of 16
    ([40], [500], 40, 1),                                # one kv head, a group of 40
    ([300, 257], [300, 800], 4, 4),                      # a kv head each
    ([6], [900], 128, 1),                                # a group of 128
    ([700, 90], [1500, 90], 14, 2),                      # a group of 7, several blocks of rows
]


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_chunk(shape, dtype, dim):
    ql, kl, heads, kv = SHAPES[shape]
    b = Batch(ql, kl, heads, kv, dim, dtype, seed=shape)
    b.check(b.attend(), b.reference())


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (63, 0), (64, 4), (65, 64), (100, 130), (128, 1),
                                          (300, 70), (5000, 4), (2 ** 31 - 1, 0)])
@pytest.mark.parametrize("shape,dtype,dim", [(1, BF, 128), (3, FP, 64), (4, BF, 64), (5, FP, 128),
                                             (6, FP, 128), (7, BF, 128), (9, FP, 64), (11, BF, 128)])
def test_window_and_sinks(shape, dtype, dim, window, sinks):
    ql, kl, heads, kv = SHAPES[shape]
    b = Batch(ql, kl, heads, kv, dim, dtype, seed=100 + shape)
    b.check(b.attend(window=window, sinks=sinks), b.reference(window=window, sinks=sinks))


@pytest.mark.parametrize("layout", ["pages", "heads", "joint"])
@pytest.mark.parametrize("shape", [3, 6])
def test_layouts_and_strides(shape, layout):
    ql, kl, heads, kv = SHAPES[shape]
    b = Batch(ql, kl, heads, kv, 64, BF, seed=7, layout=layout, q_pad=8)
    want = b.reference(window=90, sinks=5)
    b.check(b.attend(window=90, sinks=5), want)
    wide = torch.full((b.table.shape[0], b.width + 5), -1, dtype=torch.int32, device=DEV)
    wide[:, :b.width] = b.table
    b.table = wide[:, :b.width]
    b.check(b.attend(window=90, sinks=5), want)


@pytest.mark.parametrize("hint", [0, 1, 100000])
def test_query_length_hint_changes_nothing_but_speed(hint):
    b = Batch([1, 40, 9, 300], [300, 60, 9, 1000], 16, 2, 128, BF, seed=3)
    b.check(b.attend(max_query_len=hint), b.reference())


def test_scale_and_large_scores():
    b = Batch([3, 200], [300, 500], 8, 2, 128, FP, seed=4)
    for scale in (1e-4, 0.5, 4.0):
        b.check(b.attend(scale=scale), b.reference(scale=scale))


@pytest.mark.parametrize("ql,kl", [([1] * 4, [40000, 3, 9000, 17000]), ([500, 1], [20000, 20000])])
def test_long_rows_split_over_ctas(ql, kl):
    b = Batch(ql, kl, 8, 1, 128, BF, seed=5)
    b.check(b.attend(), b.reference())
    b.check(b.attend(window=15000, sinks=100), b.reference(window=15000, sinks=100))


def test_many_requests():
    g = torch.Generator().manual_seed(1)
    kl = torch.randint(0, 130, (1500,), generator=g).tolist()
    b = Batch([1] * 1500, kl, 4, 2, 64, FP, seed=6)
    b.check(b.attend(), b.reference())


@pytest.mark.parametrize("ql,kl", [([2, 40], [130, 200]), ([260, 140], [260, 400])])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_nonfinite_values_reach_only_rows_that_see_them(ql, kl, dtype):
    """A later token's infinities and NaNs, or a token's that has left the window, must not
    reach the rows that do not see it (a weight of 0 times an infinity is a NaN)."""
    b = Batch(ql, kl, 8, 2, 128, dtype, seed=8)
    clean, _ = b.attend(window=70, sinks=2)
    for key, value in ((kl[0] - 1, float("nan")), (kl[0] - 2, float("inf")), (kl[0] - 72, float("-inf"))):
        page, slot = int(b.table[0, key // PAGE]), key % PAGE
        for cache in (b.v, b.k):
            keep = cache[page, slot].clone()
            cache[page, slot] = value
            out, _ = b.attend(window=70, sinks=2)
            cache[page, slot] = keep
            pos = torch.arange(ql[0], device=DEV) + (kl[0] - ql[0])
            see = (key <= pos) & ((pos - key < 70) | (key < 2))
            rows = torch.ones(b.rows, dtype=torch.bool, device=DEV)
            rows[:ql[0]] = ~see
            assert torch.equal(out[rows], clean[rows])
            if cache is b.v:
                assert not torch.isfinite(out[~rows]).any()


def test_results_do_not_depend_on_timing():
    b = Batch([1] * 8 + [150], [5000] * 8 + [900], 16, 2, 128, BF, seed=9)
    first = b.attend()
    for _ in range(5):
        again = b.attend()
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def _lists(b, topk, empty_rows=()):
    """Distinct positions each row may see, in no order, then -1 at random places."""
    rows = []
    for r, (nq, n) in enumerate(zip(b.ql, b.kl)):
        for i in range(nq):
            seen = max(0, n - nq + i + 1)
            take = min(topk, seen)
            if len(rows) in empty_rows:
                take = 0
            row = torch.full((topk,), -1, dtype=torch.int64, device=DEV)
            where = torch.randperm(topk, generator=b.gen, device=DEV)[:take]
            row[where] = torch.randperm(max(1, seen), generator=b.gen, device=DEV)[:take]
            rows.append(row)
    return torch.stack(rows).to(torch.int32)


@pytest.mark.parametrize("topk", [1, 15, 64, 200, 2048])
@pytest.mark.parametrize("shape,dtype,dim", [(1, BF, 128), (2, FP, 64), (3, BF, 64), (4, FP, 128), (7, BF, 128),
                                             (8, BF, 64), (9, FP, 128), (10, FP, 64)])
def test_selected(shape, dtype, dim, topk):
    ql, kl, heads, kv = SHAPES[shape]
    b = Batch(ql, kl, heads, kv, dim, dtype, seed=200 + shape)
    idx = _lists(b, topk, empty_rows=(1,))
    b.check(b.attend_selected(idx), b.reference(indices=idx))


def test_selected_repeats_and_strided_lists():
    b = Batch([1, 3], [300, 90], 8, 2, 64, BF, seed=11)
    idx = torch.randint(0, 80, (4, 96), generator=b.gen, device=DEV, dtype=torch.int32)
    wide = torch.zeros((4, 130), dtype=torch.int32, device=DEV)
    wide[:, :96] = idx
    b.check(b.attend_selected(wide[:, :96]), b.reference(indices=idx))


def test_selected_long_lists_agree_with_causal_rows():
    """A list of every key gives what the causal form gives to within both tolerances."""
    b = Batch([1] * 3, [2000, 700, 2048], 16, 2, 128, BF, seed=12)
    idx = torch.full((3, 2048), -1, dtype=torch.int32, device=DEV)
    for r, n in enumerate(b.kl):
        idx[r, :n] = torch.randperm(n, generator=b.gen, device=DEV).to(torch.int32)
    want = b.reference()
    b.check(b.attend_selected(idx), want)
    b.check(b.attend(), want)


def test_rows_outside_every_request_are_left_alone():
    b = Batch([2, 3], [70, 80], 4, 2, 64, BF, seed=13)
    want = b.reference()
    q = torch.zeros((9, 4, 64), dtype=BF, device=DEV)
    q[2:7] = b.q
    start = b.start + 2
    idx = torch.full((9, 128), -1, dtype=torch.int32, device=DEV)
    for selected in (False, True):
        out, lse = torch.full_like(q, 7.0), torch.full((9, 4), 7.0, device=DEV)
        if selected:
            for r, seen in zip(range(2, 7), [69, 70, 78, 79, 80]):
                idx[r, :seen] = torch.arange(seen, device=DEV, dtype=torch.int32)
            saib.indexer_attend_selected(q, b.k, b.v, b.table, idx, start, out=out, lse=lse)
        else:
            saib.indexer_attend_paged(q, b.k, b.v, b.table, b.lens, start, 3, out=out, lse=lse)
        torch.cuda.synchronize()
        assert (out[:2] == 7).all() and (out[7:] == 7).all() and (lse[7:] == 7).all()
        b.check((out[2:7], lse[2:7]), want)


def test_bad_lengths_and_pages_are_reported():
    b = Batch([1, 1], [100, 100], 4, 2, 64, BF, seed=14)
    want = b.reference()
    cases = [("lens", torch.tensor([100, b.width * 64 + 1], dtype=torch.int32, device=DEV), 2 | 1),
             ("lens", torch.tensor([100, -3], dtype=torch.int32, device=DEV), 2),
             ("start", torch.tensor([0, 1, 9], dtype=torch.int32, device=DEV), 2)]
    table = b.table.clone()
    table[1, 1] = b.k.shape[0]
    cases.append(("table", table, 1))
    for name, value, bits in cases:
        keep = getattr(b, name)
        setattr(b, name, value)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        out, lse = saib.indexer_attend_paged(b.q, b.k, b.v, b.table, b.lens, b.start, 1, dev_error=err)
        torch.cuda.synchronize()
        setattr(b, name, keep)
        assert int(err.item()) & bits and not int(err.item()) & ~bits, (name, int(err.item()))
        assert ((out[0].double() - want[0][0]).abs() <= want[2][0]).all()   # the sound request
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    idx = torch.tensor([[5, 6], [b.width * 64, 7]], dtype=torch.int32, device=DEV)
    out, _ = saib.indexer_attend_selected(b.q, b.k, b.v, b.table, idx, b.start, dev_error=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 1 and torch.isfinite(out).all()


def test_graph_capture_and_other_streams():
    b = Batch([1, 150, 2], [500, 400, 70], 8, 2, 128, BF, seed=15)
    want = b.reference(window=200, sinks=3)
    idx = _lists(b, 100)
    want_sel = b.reference(indices=idx)
    ws = saib.attend_workspace(b.rows, 3, 8, 2, 128, DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        got = saib.indexer_attend_paged(b.q, b.k, b.v, b.table, b.lens, b.start, 150, window=200, sinks=3,
                                        stream=stream)
        side.synchronize()
        b.check(got, want)
    out, lse = torch.empty_like(b.q), torch.empty((b.rows, 8), device=DEV)
    out2, lse2 = torch.empty_like(out), torch.empty_like(lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        saib.indexer_attend_paged(b.q, b.k, b.v, b.table, b.lens, b.start, 150, window=200, sinks=3, out=out,
                                  lse=lse, workspace=ws)
        saib.indexer_attend_selected(b.q, b.k, b.v, b.table, idx, b.start, out=out2, lse=lse2, workspace=ws)
    for _ in range(3):
        for t in (out, lse, out2, lse2):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        b.check((out, lse), want)
        b.check((out2, lse2), want_sel)


def test_offsets_past_32_bits():
    """A cache of more than 2^31 elements: pages at both of its ends."""
    pages = (1 << 31) // (PAGE * 8 * 128) + 40
    k = torch.zeros((pages, PAGE, 8, 128), dtype=BF, device=DEV)
    v = torch.zeros_like(k)
    b = Batch([1, 130], [200, 300], 16, 8, 128, BF, seed=16, extra_pages=0)
    n = b.k.shape[0]
    k[-n:], v[-n:] = b.k, b.v
    want = b.reference()
    b.table = torch.where(b.table >= 0, b.table + (pages - n), b.table)
    b.k, b.v = k, v
    b.check(b.attend(), want)
    idx = _lists(b, 64)
    ref = b.reference(indices=idx)
    b.check(b.attend_selected(idx), ref)


# ---- more of the chunk kernel's (over 16 rows a kv head) and the many-token lists' edges


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("ql,kl,heads,kv", [
    ([200, 0, 90, 1], [150, 10, 0, 500], 8, 2),          # fewer keys than tokens, no tokens, no keys
    ([0, 0, 257, 0], [5, 0, 257, 9], 16, 2),
    ([17, 33, 64, 65], [17, 4000, 64, 191], 16, 16),     # a kv head each: units of few rows
    ([128, 129], [128, 1290], 2, 1),                     # exactly one block of 256 rows, and two rows more
    ([1, 1, 1, 500], [3000, 1, 0, 640], 24, 2),          # single tokens beside a chunk
])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 3), (1, 200)])
def test_chunk_batches(ql, kl, heads, kv, window, sinks, dim):
    b = Batch(ql, kl, heads, kv, dim, BF, seed=31)
    b.check(b.attend(window=window, sinks=sinks), b.reference(window=window, sinks=sinks))


@pytest.mark.parametrize("ql,kl", [([1, 2], [300, 70]), ([150, 3], [400, 70])])
def test_padded_caches(ql, kl):
    """Pages with slack between tokens, heads and pages: strides that are multiples of 8 values and
    of nothing else; and a cache of one head shared by all (a stride of 0)."""
    b = Batch(ql, kl, 8, 2, 64, FP, seed=32)
    want = b.reference()
    pages = b.k.shape[0]
    for cache in ("k", "v"):
        wide = torch.full((pages * (65 * 2 * 72) + 8,), float("nan"), dtype=FP, device=DEV)
        view = wide[8:].as_strided((pages, PAGE, 2, 64), (65 * 2 * 72 - 8 * (cache == "k"), 2 * 72, 72, 1))
        view.copy_(getattr(b, cache))
        setattr(b, cache, view)
    b.check(b.attend(), want)
    idx = _lists(b, 30)
    b.check(b.attend_selected(idx), b.reference(indices=idx))
    b.k, b.v = b.k[:, :, :1].expand(-1, -1, 2, -1), b.v[:, :, :1].expand(-1, -1, 2, -1)
    assert b.k.stride(2) == 0
    b.check(b.attend(window=50, sinks=1), b.reference(window=50, sinks=1))


def test_chunk_rows_outside_every_request_are_left_alone():
    b = Batch([60, 30], [100, 80], 8, 2, 64, BF, seed=33)
    want = b.reference()
    q = torch.zeros((100, 8, 64), dtype=BF, device=DEV)
    q[4:94] = b.q
    out, lse = torch.full_like(q, 7.0), torch.full((100, 8), 7.0, device=DEV)
    saib.indexer_attend_paged(q, b.k, b.v, b.table, b.lens, b.start + 4, 60, out=out, lse=lse)
    torch.cuda.synchronize()
    assert (out[:4] == 7).all() and (out[94:] == 7).all() and (lse[:4] == 7).all() and (lse[94:] == 7).all()
    b.check((out[4:94], lse[4:94]), want)


def test_chunk_reports_bad_lengths_and_pages():
    b = Batch([60, 30], [200, 180], 8, 2, 64, BF, seed=34)
    want = b.reference()
    table = b.table.clone()
    table[1, 1] = b.k.shape[0]
    cases = [("lens", torch.tensor([200, b.width * 64 + 1], dtype=torch.int32, device=DEV), 2 | 1),
             ("lens", torch.tensor([200, -3], dtype=torch.int32, device=DEV), 2),
             ("start", torch.tensor([0, 60, 990], dtype=torch.int32, device=DEV), 2),
             ("start", torch.tensor([0, 60, 20], dtype=torch.int32, device=DEV), 2),
             ("table", table, 1)]
    for name, value, bits in cases:
        keep = getattr(b, name)
        setattr(b, name, value)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        out, _ = saib.indexer_attend_paged(b.q, b.k, b.v, b.table, b.lens, b.start, 60, dev_error=err)
        torch.cuda.synchronize()
        setattr(b, name, keep)
        got = int(err.item())
        assert got & bits and not got & ~bits, (name, got)
        assert ((out[:60].double() - want[0][:60]).abs() <= want[2][:60]).all()   # the sound request
    b.check(b.attend(), want)


@pytest.mark.parametrize("heads,kv,topk,dtype,dim", [(8, 2, 100, BF, 128), (40, 1, 33, FP, 64), (6, 3, 17, BF, 64),
                                                    (16, 1, 260, FP, 128), (4, 4, 1, BF, 128)])
def test_lists_of_many_tokens(heads, kv, topk, dtype, dim):
    b = Batch([700, 0, 300, 5], [900, 10, 300, 3], heads, kv, dim, dtype, seed=35)
    idx = _lists(b, topk, empty_rows=(0, 3, 699, 700, 1004))
    b.check(b.attend_selected(idx), b.reference(indices=idx))


def test_lists_of_many_tokens_outside_requests_and_bad_entries():
    b = Batch([400, 300], [500, 300], 4, 2, 64, BF, seed=36)
    idx = _lists(b, 20)
    want = b.reference(indices=idx)
    q = torch.zeros((900, 4, 64), dtype=BF, device=DEV)
    q[100:800] = b.q
    lists = torch.full((900, 20), 3, dtype=torch.int32, device=DEV)
    lists[100:800] = idx
    out, lse = torch.full_like(q, 7.0), torch.full((900, 4), 7.0, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    saib.indexer_attend_selected(q, b.k, b.v, b.table, lists, b.start + 100, out=out, lse=lse, dev_error=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert (out[:100] == 7).all() and (out[800:] == 7).all() and (lse[:100] == 7).all() and (lse[800:] == 7).all()
    b.check((out[100:800], lse[100:800]), want)
    lists[100, 4] = b.width * PAGE          # past the table
    lists[799, 0] = 5 * PAGE                # an unused column: page -7
    saib.indexer_attend_selected(q, b.k, b.v, b.table, lists, b.start + 100, out=out, lse=lse, dev_error=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 1
    b.check((out[101:799], lse[101:799]), tuple(w[1:699] for w in want))
