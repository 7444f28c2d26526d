"""Appends to the paged key/value cache with the rotation, and MXFP4 index-key inserts, on the GPU.

Tolerance of a rotated value a c - b s (u = half a step of the type, eps / 2): two fp32
roundings of at most 2^-24 of |a c| + |b s| each, then one to the type: u of the value, or 2^-25 where
fp16 is subnormal. Values that are moved, and MXFP4 entries (divisions by powers of two are
exact), are equal bit for bit.
"""
import numpy as np
import pytest
import torch

import oracle
import synth
import sparse_attention_indexer_block_gb300 as saib
from test_gpu_attend import BF, DEV, FP, PAGE, _lib  # noqa: F401

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _table(positions, rotary_dim, g):
    angle = torch.rand((positions, rotary_dim // 2), generator=g, device=DEV, dtype=torch.float64) * 6.2832
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _rotated(x, positions, rotary, interleaved):
    """(x rotated in 64 bits, its tolerance)."""
    u = torch.finfo(x.dtype).eps / 2
    x = x.double()
    half = rotary.shape[1] // 2
    row = rotary.double()[positions.long()]
    c, s = row[:, None, :half], row[:, None, half:]
    if interleaved:
        ia, ib = torch.arange(0, 2 * half, 2, device=DEV), torch.arange(1, 2 * half, 2, device=DEV)
    else:
        ia, ib = torch.arange(half, device=DEV), torch.arange(half, 2 * half, device=DEV)
    a, b = x[..., ia], x[..., ib]
    out, tol = x.clone(), torch.zeros_like(x)
    out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
    tol[..., ia] = 2.0 ** -23 * ((a * c).abs() + (b * s).abs())
    tol[..., ib] = 2.0 ** -23 * ((b * c).abs() + (a * s).abs())
    turned = torch.zeros(x.shape[-1], dtype=torch.bool, device=DEV)
    turned[:2 * half] = True
    tol = torch.where(turned, tol * (1 + u) + u * out.abs() + 2.0 ** -25, 0.0)
    return out, tol


def _close(got, want):
    out, tol = want
    bad = (got.double() - out).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} values, first {bad.nonzero()[0].tolist()}"


class Append:
    def __init__(self, tokens, heads, kv, dim, dtype, rotary_dim, seed=0, pages=None, layout="pages", positions=5000):
        g = _gen(seed)
        self.kv, self.dim = kv, dim
        pages = pages or -(-tokens // PAGE) + 3
        qkv = torch.randn((tokens, (heads + 2 * kv) * dim), generator=g, device=DEV).to(dtype)
        self.q = qkv[:, :heads * dim].view(tokens, heads, dim)
        self.k = qkv[:, heads * dim:(heads + kv) * dim].view(tokens, kv, dim)
        self.v = qkv[:, (heads + kv) * dim:].view(tokens, kv, dim)
        both = torch.randn((pages, 2, PAGE, kv, dim), generator=g, device=DEV).to(dtype)
        self.k_cache, self.v_cache = both[:, 0].contiguous(), both[:, 1].contiguous()
        if layout == "heads":
            self.k_cache, self.v_cache = (c.transpose(1, 2).contiguous().transpose(1, 2)
                                          for c in (self.k_cache, self.v_cache))
        elif layout == "joint":
            self.k_cache, self.v_cache = both[:, 0], both[:, 1]
        self.slots = torch.randperm(pages * PAGE, generator=g, device=DEV)[:tokens]
        self.positions = torch.randint(0, positions, (tokens,), generator=g, device=DEV, dtype=torch.int32)
        self.rotary = _table(positions, rotary_dim, g) if rotary_dim else None
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def run(self, interleaved=False, q=True, **kw):
        if self.rotary is not None:
            kw.update(positions=self.positions, rotary=self.rotary, interleaved=interleaved)
            if q:
                kw.update(q=self.q)
        out = saib.indexer_append_kv(self.k, self.v, self.k_cache, self.v_cache, self.slots, dev_error=self.err, **kw)
        torch.cuda.synchronize()
        return out

    def check(self, q_out, before, interleaved=False, valid=None, positions=None):
        valid = torch.ones_like(self.slots, dtype=torch.bool) if valid is None else valid
        positions = self.positions if positions is None else positions
        k = (self.k.double(), torch.zeros(1, device=DEV, dtype=torch.float64))
        if self.rotary is not None:
            k = _rotated(self.k, positions, self.rotary, interleaved)
        s = self.slots[valid]
        _close(self.k_cache[s // PAGE, s % PAGE], (k[0][valid], k[1][valid] if k[1].dim() > 1 else k[1]))
        assert torch.equal(self.v_cache[s // PAGE, s % PAGE], self.v[valid])
        other = torch.ones(self.k_cache.shape[:2], dtype=torch.bool, device=DEV)
        other[s // PAGE, s % PAGE] = False
        for cache, old in zip((self.k_cache, self.v_cache), before):
            assert torch.equal(cache[other], old[other])
        if q_out is not None:
            _close(q_out, _rotated(self.q, positions, self.rotary, interleaved))

    def before(self):
        return self.k_cache.clone(), self.v_cache.clone()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,heads,kv,dim,dtype,rotary_dim", [
    (1, 32, 8, 128, BF, 128), (1, 1, 1, 64, FP, 64), (33, 5, 1, 128, FP, 64), (130, 64, 8, 128, BF, 128),
    (7, 48, 3, 64, BF, 16), (500, 12, 4, 64, FP, 64), (65, 128, 1, 128, BF, 112), (1, 3, 3, 128, BF, 16),
    (3001, 6, 2, 128, FP, 32), (2500, 40, 8, 64, BF, 48)])
def test_append(tokens, heads, kv, dim, dtype, rotary_dim, interleaved):
    a = Append(tokens, heads, kv, dim, dtype, rotary_dim, seed=tokens)
    old = a.before()
    out = a.run(interleaved)
    a.check(out, old, interleaved)
    assert int(a.err) == 0


@pytest.mark.parametrize("layout", ["pages", "heads", "joint"])
@pytest.mark.parametrize("rotary_dim", [0, 64])
def test_append_layouts_and_no_queries(layout, rotary_dim):
    a = Append(90, 4, 3, 64, BF, rotary_dim, seed=1, layout=layout)
    old = a.before()
    assert a.run(q=False) is None
    a.check(None, old)


def test_append_in_place_and_strided_queries():
    a = Append(70, 8, 2, 128, FP, 96, seed=2)
    q = a.q.clone()
    want = _rotated(a.q, a.positions, a.rotary, False)
    out = a.run(q_out=a.q)
    assert out is a.q
    _close(a.q, want)
    wide = torch.full((70, 8, 136), 7.0, device=DEV, dtype=FP)
    a.q = q
    assert a.run(q_out=wide[:, :, :128]) is not None
    _close(wide[:, :, :128], want)
    assert (wide[:, :, 128:] == 7).all()


def test_append_padding_bad_slots_and_positions():
    a = Append(40, 4, 2, 64, BF, 64, seed=3, positions=100)
    slots, positions = a.slots.clone(), a.positions.clone()
    valid = torch.ones(40, dtype=torch.bool, device=DEV)
    # padding, with a position that is nowhere
    a.slots[37:] = -1
    a.positions[39] = 1 << 30
    valid[37:] = False
    old = a.before()
    out = a.run()
    assert int(a.err) == 0
    a.check(out, old, valid=valid, positions=a.positions.clamp(0, 99))
    # slots past the cache
    a.slots, a.positions = slots.clone(), positions.clone()
    a.slots[3], a.slots[9] = a.k_cache.shape[0] * PAGE, 1 << 40
    valid[:] = True
    valid[3] = valid[9] = False
    old = a.before()
    out = a.run()
    assert int(a.err) == 1
    a.check(out, old, valid=valid)
    # positions outside the table are clamped
    a.slots, a.err[0] = slots, 0
    a.positions[5], a.positions[6] = -4, 100
    old = a.before()
    out = a.run()
    assert int(a.err) == 2
    a.check(out, old, positions=a.positions.clamp(0, 99))


def test_append_nothing():
    a = Append(4, 4, 2, 64, BF, 64, seed=4)
    old = a.before()
    a.k, a.v, a.q, a.slots, a.positions = a.k[:0], a.v[:0], a.q[:0], a.slots[:0], a.positions[:0]
    assert a.run().shape == (0, 4, 64)
    assert torch.equal(a.k_cache, old[0]) and torch.equal(a.v_cache, old[1])


def test_append_nonfinite_values_stay_in_their_pairs():
    a = Append(3, 2, 1, 128, BF, 64, seed=5)
    a.k[0, 0, 3], a.k[1, 0, 100], a.v[2, 0, 5] = float("inf"), float("nan"), float("nan")
    a.run()
    s = a.slots
    k, v = a.k_cache[s // PAGE, s % PAGE], a.v_cache[s // PAGE, s % PAGE]
    odd = ~torch.isfinite(k[:, 0])
    assert set(map(tuple, odd.nonzero().tolist())) == {(0, 3), (0, 35), (1, 100)}
    assert torch.isnan(v).nonzero().tolist() == [[2, 0, 5]]


def test_append_far_offsets():
    """Slots whose values lie past 2^31 elements."""
    pages = 2 ** 31 // (PAGE * 8 * 128) + 40
    a = Append(5, 8, 8, 128, BF, 128, seed=6, pages=1)
    a.k_cache = torch.zeros((pages, PAGE, 8, 128), dtype=BF, device=DEV)
    a.v_cache = torch.zeros_like(a.k_cache)
    a.slots = torch.tensor([0, pages * PAGE - 1, pages * PAGE - 2, 2 ** 31 // 1024, 2 ** 31 // 1024 - 1], device=DEV)
    a.run()
    assert int(a.err) == 0
    k, v = (c[a.slots // PAGE, a.slots % PAGE] for c in (a.k_cache, a.v_cache))
    _close(k, _rotated(a.k, a.positions, a.rotary, False))
    assert torch.equal(v, a.v)
    assert int((a.v_cache != 0).any(-1).sum()) == 5 * 8


# ---------------------------------------------------------------------------
# MXFP4 index keys
# ---------------------------------------------------------------------------


def _keys(n, seed):
    g = _gen(seed)
    k = torch.randn((n, 128), generator=g, device=DEV) * torch.exp(3 * torch.randn((n, 1), generator=g, device=DEV))
    return k.to(BF)


@pytest.mark.parametrize("tokens", [1, 2, 7, 64, 1001, 40000])
def test_insert_mxfp4(tokens):
    k = _keys(tokens, tokens)
    if tokens > 1:
        k[0] = 0
        k[1, :32] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.0, 6.0, 7.0, -7.9, 0.0, -0.0, -0.1, 4.0,
                                  4.5] * 2, device=DEV)
    pages = -(-tokens // PAGE) + 2
    slots = torch.randperm(pages * PAGE, generator=_gen(1), device=DEV)[:tokens]
    cache = torch.full((pages, 4352), 0xaa, dtype=torch.uint8, device=DEV)
    values = torch.empty_like(k)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    assert saib.indexer_insert_keys_mxfp4(k, slots, cache, values=values, dev_error=err) is cache
    torch.cuda.synchronize()
    assert int(err) == 0
    want = oracle.mxfp4_quantize(k.float().cpu().numpy())
    got = cache.view(-1, 68)
    assert np.array_equal(got[slots].cpu().numpy(), want)
    other = torch.ones(pages * PAGE, dtype=torch.bool, device=DEV)
    other[slots] = False
    assert (got[other] == 0xaa).all()
    assert np.array_equal(values.double().cpu().numpy(), oracle.mxfp4_values(want))


def test_insert_mxfp4_extremes():
    """Blocks of subnormals, of the largest values, with infinities and NaNs."""
    tiny = torch.finfo(BF).tiny
    k = torch.zeros((6, 128), dtype=BF, device=DEV)
    k[0, :8] = torch.tensor([tiny, tiny / 2, tiny / 128, -tiny / 4, 3 * tiny, 0, tiny / 64, tiny / 16], device=DEV)
    k[1, :4] = torch.tensor([3.3e38, -1e38, 1e30, 2e38], device=DEV)
    k[2, 40:44] = torch.tensor([2.0 ** -126, 2.0 ** -125, 2.0 ** -124, -2.0 ** -123], device=DEV)
    k[3, 64:66] = torch.tensor([float("nan"), 1.0], device=DEV)
    k[4, 96:99] = torch.tensor([float("-inf"), 3e38, 1.0], device=DEV)
    k[5, :2] = torch.tensor([float("nan"), float("nan")], device=DEV)
    cache = torch.zeros((1, 4352), dtype=torch.uint8, device=DEV)
    values = torch.empty_like(k)
    slots = torch.arange(6, device=DEV)
    saib.indexer_insert_keys_mxfp4(k, slots, cache, values=values)
    torch.cuda.synchronize()
    got = cache.view(-1, 68)[:6].cpu().numpy()
    plain = torch.where(k.isnan(), 0.0, k.float())
    want = oracle.mxfp4_quantize(plain[:4].cpu().numpy())
    assert np.array_equal(got[:4], want) and not got[5].any()
    assert np.array_equal(values[:4].double().cpu().numpy(), oracle.mxfp4_values(want))
    # -inf: scale 2^126, code -6; 3e38 / 2^126 = 3.5 goes to 4 (even)
    assert got[4, 67] == 253 and got[4, 48] == 0xf | 0x6 << 4 and not got[4, 49:64].any()
    assert values[4, 96] == float("-inf") and values[4, 97] == 4 * 2.0 ** 126


def test_insert_mxfp4_padding_bad_slots_and_strides():
    wide = _keys(50, 5).repeat(1, 2)[:, :160]
    k = wide[:, 16:144]
    assert k.stride(0) == 256
    slots = torch.arange(50, device=DEV) * 2
    slots[4], slots[20], slots[21] = -1, 2 * PAGE, 1 << 50
    cache = torch.full((2, 4352), 0x11, dtype=torch.uint8, device=DEV)
    values = torch.full((50, 128), 7.0, dtype=BF, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    saib.indexer_insert_keys_mxfp4(k, slots, cache, values=values, dev_error=err)
    torch.cuda.synchronize()
    assert int(err) == 1
    gone = (slots < 0) | (slots >= 2 * PAGE)
    want = oracle.mxfp4_quantize(k.float().contiguous().cpu().numpy())
    keep = ~gone.cpu().numpy()
    assert np.array_equal(cache.view(-1, 68)[slots[~gone]].cpu().numpy(), want[keep])
    assert (cache.view(-1, 68)[1::2] == 0x11).all()
    assert not values[gone].any()
    assert np.array_equal(values[~gone].double().cpu().numpy(), oracle.mxfp4_values(want[keep]))


def test_insert_mxfp4_feeds_the_selection():
    """Keys inserted here and read by the MXFP4 top-k: the logits of the oracle on the same entries."""
    m = synth.make_decode_mxfp4_from_lens([700, 130], [1, 1], 1, seed=9)
    k = _keys(830, 10)
    table, cache = m.block_table.to(DEV), torch.zeros_like(m.cache, device=DEV)
    slots = torch.cat([table[r, torch.arange(n, device=DEV) // PAGE].long() * PAGE + torch.arange(n, device=DEV) % PAGE
                       for r, n in enumerate((700, 130))])
    saib.indexer_insert_keys_mxfp4(k, slots, cache)
    logits = saib.indexer_decode_logits_mxfp4(m.q.to(DEV), m.w.to(DEV), cache, table, m.seq_lens.to(DEV))
    torch.cuda.synchronize()
    q8, _, wp = oracle.quantize_q(synth.bf16_bits(m.q), m.w.numpy())
    for r, n in enumerate((700, 130)):
        o, a, b = oracle.row_logits_mxfp4(q8[r], wp[r], cache.cpu().numpy(), m.block_table.numpy()[r], n)
        got = logits[r, :n].double().cpu().numpy()
        assert (np.abs(got - o) <= 1e-3 * a + 1e-5 * b).all()
