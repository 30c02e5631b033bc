"""The paged 4-bit cache and rotary positions without a GPU: the oracle's own pins, the binding's helpers, and the
refusals of the C entry points and of the binding (none of which makes a CUDA call)."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import paged


# ----------------------------------------------------------------------------------------- oracle

def test_rope_is_a_complex_product_and_its_inverse_undoes_it():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 3, 12))
    pos = np.array([0, 1, 7, 100000, -4])
    f = np.array([1.0, 0.1, 0.003])
    for inter in (False, True):
        y = paged.rope_rotate(x, pos, f, first=4, interleaved=inter, gain=1.5)
        np.testing.assert_array_equal(y[..., :4], x[..., :4])
        np.testing.assert_array_equal(y[..., 10:], x[..., 10:])
        v = x[..., 4:10]
        z = v[..., 0::2] + 1j * v[..., 1::2] if inter else v[..., :3] + 1j * v[..., 3:]
        w = 1.5 * z * np.exp(1j * pos[:, None, None] * f)
        got = y[..., 4:10]
        g = got[..., 0::2] + 1j * got[..., 1::2] if inter else got[..., :3] + 1j * got[..., 3:]
        np.testing.assert_allclose(g, w, atol=1e-12)
        back = paged.rope_rotate(y, pos, f, first=4, interleaved=inter, inverse=True, gain=1 / 1.5)
        np.testing.assert_allclose(back, x, atol=1e-12)


def test_rope_scores_depend_on_the_distance_alone():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((1, 1, 8)), rng.standard_normal((1, 1, 8))
    f = 10000.0 ** (-np.arange(4) / 4)
    dot = lambda a, b: float((paged.rope_rotate(q, [a], f) * paged.rope_rotate(k, [b], f)).sum())  # noqa: E731
    assert abs(dot(17, 5) - dot(1012, 1000)) < 1e-10
    assert abs(dot(17, 5) - dot(17, 6)) > 1e-3


@pytest.mark.parametrize("amax,want", [(7.0, 8 / 8), (7.03125, 9 / 8), (105.0, 15), (105.5, 16), (0.0, 0), (2.0 ** -101, 0),
                                       (56.0, 8), (112.0, 16), (1.0, 10 / 64)])
def test_block_scale_closed_forms(amax, want):
    assert paged.block_scale(amax) == Fraction(want)


def test_codes_round_to_nearest_even_and_fill_the_range():
    x = np.zeros((1, 32), dtype=np.float32)
    x[0, :8] = [7, 0.5, 1.5, 2.5, -0.5, -1.5, 3.49, -7]
    codes, scales = paged.quantize_rows(x)
    assert scales[0, 0] == 1.0
    assert codes[0, :8].tolist() == [7, 0, 2, 2, 0, -2, 3, -7]
    rng = np.random.default_rng(2)
    v = torch.from_numpy(rng.standard_normal((50, 64)).astype(np.float32)).bfloat16()
    codes, scales = paged.quantize_rows(v)
    assert np.abs(codes).max() == 7
    held = codes * np.repeat(scales, 32, axis=1)
    assert np.abs(held - v.float().numpy()).max() <= scales.max() / 2          # half a step
    np.testing.assert_array_equal(held, torch.from_numpy(held).bfloat16().double().numpy())   # exact in bf16


def test_pack_round_trip_and_bit_places():
    rng = np.random.default_rng(3)
    codes = rng.integers(-8, 8, (5, 96))
    np.testing.assert_array_equal(paged.unpack_codes(paged.pack_codes(codes)), codes)
    one = np.full((1, 32), -8)
    one[0, 3] = 7          # column 3: the upper half's second nibble
    w = paged.pack_codes(one).view(np.uint32)[0]
    assert w[0] == 15 << 20 and (w[1:] == 0).all()


def test_paged_decode_oracle_equals_the_contiguous_one():
    import oracle
    from paged_util import bits, make_pool, queries
    rng = np.random.default_rng(4)
    lens, G, d, page = [5, 9, 2], 2, 128, 4
    pool, table = make_pool(rng, lens, G, d, page)
    q, qr = queries(rng, 3, 2, 6, d)
    out, lse, spread, _ = paged.paged_decode(q, qr, pool, G, table, lens, 0.07)
    rows = np.concatenate([np.stack([pool[table[b, t // page], t % page] for t in range(n)]) for b, n in enumerate(lens)])
    r = G * d
    sc = torch.from_numpy(rows[:, r // 2:r // 2 + r // 16].copy()).view(torch.bfloat16).double().numpy()
    lat = paged.unpack_codes(rows[:, :r // 2]) * np.repeat(sc, 32, axis=1)
    kpe = torch.from_numpy(rows[:, -128:].copy()).view(torch.bfloat16)
    w_out, w_lse = oracle.gta_group_decode(q, qr, torch.from_numpy(lat), kpe, G, np.array([0, 5, 14, 16]), 0.07)
    np.testing.assert_allclose(out, w_out, atol=1e-12)
    np.testing.assert_allclose(lse, w_lse, atol=1e-12)
    assert (spread >= np.abs(out) - 1e-15).all() and bits(kpe).shape == (16, 64)


# ---------------------------------------------------------------------------------------- helpers

def test_row_bytes(lkv_built):
    L = lkv_built
    for r, dr, want in [(1024, 64, 704), (512, 64, 416), (256, 64, 272), (128, 64, 208), (32, 0, 32), (64, 8, 64)]:
        assert L.int4_cache_row_bytes(r, dr) == want == paged.row_bytes(r, dr)
    for r, dr in [(0, 64), (48, 64), (1056, 64), (512, 4), (512, -8), (512, 1032)]:
        assert L.int4_cache_row_bytes(r, dr) == 0


def test_fields_are_views_of_the_rows(lkv_built):
    rng = np.random.default_rng(5)
    r, dr = 320, 16
    codes = rng.integers(-7, 8, (6, r))
    scales = rng.integers(8, 16, (6, r // 32)) / 64
    key = rng.integers(0, 1 << 15, (6, dr)).astype(np.uint16)
    rows = paged.pack_rows(codes, scales, key, dr)
    pool = torch.zeros((2, 3, rows.shape[1] + 32), dtype=torch.uint8)
    pool[..., :rows.shape[1]] = torch.from_numpy(rows).view(2, 3, -1)
    c, s, k = lkv_built.int4_cache_fields(pool, r, dr)
    np.testing.assert_array_equal(paged.unpack_codes(c.numpy()).reshape(6, r), codes)
    np.testing.assert_array_equal(s.float().numpy().reshape(6, -1), scales)
    np.testing.assert_array_equal(k.contiguous().view(torch.int16).numpy().view(np.uint16).reshape(6, dr), key)
    with pytest.raises(ValueError):
        lkv_built.int4_cache_fields(pool[..., :100], r, dr)


def test_rope_frequencies(lkv_built):
    f, gain = lkv_built.rope_frequencies(8)
    assert gain == 1.0 and f.dtype == torch.float64
    np.testing.assert_allclose(f.numpy(), [1, 1e-1, 1e-2, 1e-3], rtol=1e-14)
    f, gain = lkv_built.rope_frequencies(64, factor=4.0, context=4096, beta_fast=32.0, beta_slow=1.0)
    plain, _ = lkv_built.rope_frequencies(64)
    turns = 4096 * plain / (2 * math.pi)
    assert gain == 1 + 0.1 * math.log(4)
    assert torch.equal(f[turns >= 32], plain[turns >= 32])
    assert torch.allclose(f[turns <= 1], plain[turns <= 1] / 4, rtol=1e-15)
    mid = (turns > 1) & (turns < 32)
    assert ((f[mid] > plain[mid] / 4) & (f[mid] < plain[mid])).all() and mid.any()
    f, _ = lkv_built.rope_frequencies(64, factor=4.0, beta_fast=math.inf)
    assert torch.allclose(f, plain / 4, rtol=1e-15)
    for bad in [dict(rot=7), dict(rot=0), dict(rot=8, factor=0.5), dict(rot=8, beta_fast=1.0), dict(rot=8, context=0)]:
        with pytest.raises(ValueError):
            lkv_built.rope_frequencies(**bad)


# --------------------------------------------------------------------------------------- refusals

GOOD = 4096  # an aligned address that no check follows


def _rope(L, **kw):
    a = dict(x=GOOD, x_ts=1024, x_hs=64, pos=GOOD, freqs=GOOD, n=4, heads=16, d=64, first=0, rot=64, inter=0, inv=0,
             gain=1.0, dtype=0, out=GOOD, o_ts=1024, o_hs=64)
    a.update(kw)
    return L._rope(*a.values(), None)


def test_rope_refusals(lkv_built):
    L = lkv_built
    for kw in [dict(x=None), dict(out=None), dict(pos=None), dict(freqs=None), dict(n=-1), dict(heads=0), dict(d=0),
               dict(rot=0), dict(rot=63), dict(rot=66), dict(first=-2), dict(first=2), dict(gain=0.0),
               dict(gain=math.nan), dict(gain=math.inf), dict(dtype=7), dict(x=GOOD + 1), dict(freqs=GOOD + 4)]:
        assert _rope(L, **kw) == L.ERR_INVALID_ARG, kw
    assert _rope(L, d=4096, rot=2048) == L.ERR_UNSUPPORTED
    assert _rope(L, n=0) == L.OK
    assert _rope(L, n=1 << 62, heads=1, d=64) == L.ERR_UNSUPPORTED


def test_in_place_needs_the_same_strides(lkv_built):
    """The same array with other strides would be written where other rows are still to be read."""
    L = lkv_built
    assert _append(L, held=GOOD, hs=584) == L.ERR_INVALID_ARG
    assert _append(L, held=GOOD, hs=576, n=0) == L.OK
    strides = dict(x=GOOD, xts=64 * 192, xhs=192, pos=GOOD, freqs=GOOD, n=8, heads=64, d=192, first=0, rot=64, inter=0, inv=0,
                   gain=1.0, dtype=L.BF16, out=GOOD, ots=64 * 192, ohs=192)
    assert L._rope(*dict(strides, ots=65 * 192).values(), None) == L.ERR_INVALID_ARG
    assert L._rope(*dict(strides, ohs=200).values(), None) == L.ERR_INVALID_ARG
    assert L._rope(*dict(strides, n=0).values(), None) == L.OK
    assert L._rope(*dict(strides, heads=1 << 30).values(), None) == L.ERR_UNSUPPORTED


def _append(L, **kw):
    a = dict(rows=GOOD, rs=576, n=8, pool=GOOD, ps=64 * 416, prs=416, pages=10, page=64, table=GOOD, ts=4, mp=4, lens=GOOD,
             cu=GOOD, batch=4, r=512, dr=64, freqs=GOOD, inter=0, gain=1.0, held=None, hs=0)
    a.update(kw)
    return L._paged_append(*a.values(), None)


def test_append_refusals(lkv_built):
    L = lkv_built
    for kw in [dict(rows=None), dict(pool=None), dict(table=None), dict(lens=None), dict(n=-1), dict(batch=0), dict(pages=0),
               dict(page=0), dict(mp=0), dict(ts=3), dict(r=500), dict(r=2048), dict(dr=4), dict(prs=400), dict(prs=424),
               dict(ps=64 * 416 + 8), dict(ps=16), dict(rows=GOOD + 2), dict(pool=GOOD + 8), dict(rs=570), dict(rs=568),
               dict(gain=-1.0), dict(freqs=GOOD + 2), dict(held=GOOD, hs=500), dict(held=GOOD + 2, hs=576),
               dict(cu=None, n=7)]:
        assert _append(L, **kw) == L.ERR_INVALID_ARG, kw
    assert _append(L, n=1 << 31) == L.ERR_UNSUPPORTED
    assert _append(L, n=0) == L.OK


def _decode(L, **kw):
    a = dict(q=GOOD, qr=GOOD, pool=GOOD, ps=64 * 704, prs=704, pages=10, page=64, table=GOOD, ts=4, mp=4, lens=GOOD, batch=4,
             s_q=1, h=128, g=8, d=128, dr=64, scale=0.07, out=GOOD, lse=GOOD, ws=GOOD, wsb=1 << 30)
    a.update(kw)
    return L._paged_decode(*a.values(), None)


def test_decode_refusals(lkv_built):
    L = lkv_built
    for kw in [dict(q=None), dict(qr=None), dict(pool=None), dict(table=None), dict(lens=None), dict(out=None),
               dict(lse=None), dict(batch=0), dict(h=0), dict(g=0), dict(h=100), dict(scale=0.0), dict(scale=-1.0),
               dict(scale=math.nan), dict(q=GOOD + 8), dict(qr=GOOD + 2), dict(out=GOOD + 4), dict(lse=GOOD + 2),
               dict(pool=GOOD + 4), dict(prs=688), dict(prs=708), dict(pages=0), dict(page=0), dict(mp=0), dict(ts=2)]:
        assert _decode(L, **kw) == L.ERR_INVALID_ARG, kw
    for kw in [dict(s_q=3), dict(s_q=0), dict(d=64), dict(d=384, g=2, h=8), dict(dr=128), dict(d=512, g=4, h=8),
               dict(h=258, g=1, d=512, ps=64 * 416, prs=416), dict(h=264, s_q=2, g=2, d=256, ps=64 * 416, prs=416)]:
        assert _decode(L, **kw) == L.ERR_UNSUPPORTED, kw


def test_workspace_size(lkv_built):
    L = lkv_built
    assert L.paged_decode_workspace_size(64, 2, 128, 8, 128, 148) > 0
    for a in [(0, 1, 128, 8, 128, 148), (1, 0, 128, 8, 128, 148), (1, 1, 100, 8, 128, 148), (1, 1, 128, 8, 0, 148),
              (1, 1, 128, 8, 128, 0)]:
        assert L.paged_decode_workspace_size(*a) == 0


def test_binding_refuses_before_the_call(lkv_built):
    L = lkv_built
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    pos, f = torch.zeros(4, dtype=torch.int32), torch.zeros(32, dtype=torch.float64)
    with pytest.raises(ValueError):
        L.rope_rotate(x, pos, f)                                  # not on a GPU
    with pytest.raises(TypeError):
        L.rope_rotate(x, pos.long(), f)
    with pytest.raises(TypeError):
        L.rope_rotate(x, pos, f.float())
    with pytest.raises(TypeError):
        L.rope_rotate(x, pos, f, out=x.float())
    lens, table = torch.ones(2, dtype=torch.int32), torch.zeros((2, 3), dtype=torch.int32)
    pool = torch.zeros((4, 16, 704), dtype=torch.uint8)
    rows = torch.zeros((4, 1088), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        L.paged_append_int4(rows.float(), pool, 1024, table, lens)
    with pytest.raises(TypeError):
        L.paged_append_int4(rows, pool.float(), 1024, table, lens)
    with pytest.raises(TypeError):
        L.paged_append_int4(rows, pool, 1024, table.long(), lens)
    with pytest.raises(ValueError):
        L.paged_append_int4(rows, pool, 1024, table, lens)
    q, qr = torch.zeros((2, 1, 128, 128), dtype=torch.bfloat16), torch.zeros((2, 1, 128, 64), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        L.paged_decode_int4(q.float(), qr.float(), pool, 8, table, lens, 0.07)
    with pytest.raises(TypeError):
        L.paged_decode_int4(q, qr, pool, 8, table, lens.long(), 0.07)
    with pytest.raises(ValueError):
        L.paged_decode_int4(q, qr, pool, 8, table, lens, 0.07)
