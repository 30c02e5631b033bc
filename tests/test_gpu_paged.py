"""GPU tests of rotary positions, the rotating 4-bit append and the paged 4-bit decode against the fp64 oracle
(oracle/paged.py), with the tolerances derived in paged_util.py and below."""
import math

import numpy as np
import pytest
import torch

from oracle import paged
from paged_util import D_ROPE, bits, check_decode, make_pool, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L(gpu):
    import latent_kv_cache_split_b200 as lib
    lib.check_device(clear=True)
    return lib


# ------------------------------------------------------------------------------------------- rope

def _rope_tol(x, ref, pos, freqs, first, rot, inter, gain, bf16):
    """|a cos - b sin| with cos, sin off by delta: the angle in turns is off by 3 ulp of fp64, its fraction by 2^-24 of
    itself (2 pi 2^-25 rad at most), sincospi by 4 ulp of fp32, gain * and the two products and their sum by 2^-24 each;
    then the result's own rounding."""
    v = np.abs(x[..., first:first + rot])
    a, b = (v[..., 0::2], v[..., 1::2]) if inter else (v[..., :rot // 2], v[..., rot // 2:])
    turns = np.abs(np.asarray(pos, dtype=np.float64))[:, None, None] * freqs / (2 * math.pi)
    delta = 2 * math.pi * (3 * 2.0 ** -53 * turns + 2.0 ** -25) + (4 + 4) * 2.0 ** -24
    t = gain * (a + b) * delta
    t = np.stack([t, t], -1).reshape(v.shape) if inter else np.concatenate([t, t], -1)
    tol = np.zeros_like(x)
    tol[..., first:first + rot] = t * (1 + 2.0 ** -7) + (2.0 ** -8 if bf16 else 2.0 ** -24) * np.abs(ref[..., first:first + rot])
    return tol


ROPE = [
    # tokens, heads, d, first, rot, interleaved, inverse, dtype, gain
    (1, 1, 64, 0, 64, False, False, torch.bfloat16, 1.0),
    (128, 128, 64, 0, 64, False, False, torch.bfloat16, 1.0),
    (33, 128, 192, 128, 64, True, False, torch.bfloat16, 1.0),
    (7, 5, 80, 16, 48, False, True, torch.float32, 1.25),
    (7, 5, 80, 16, 48, True, True, torch.float32, 0.5),
    (19, 3, 70, 3, 34, False, False, torch.bfloat16, 1.0),     # no 16-byte rows: one column at a time
    (19, 3, 70, 3, 34, True, False, torch.bfloat16, 1.0),
    (19, 2, 37, 1, 6, True, True, torch.float32, 1.0),
    (300, 1, 32, 0, 32, True, False, torch.float32, 1.0),      # several tokens a block
    (5, 2, 2080, 16, 1024, False, False, torch.bfloat16, 1.0),  # more items than threads, the widest table
    (5, 2, 1100, 0, 1024, True, False, torch.float32, 1.0),
    (3, 300, 64, 0, 2, False, False, torch.bfloat16, 1.0),
]


@pytest.mark.parametrize("n,h,d,first,rot,inter,inv,dtype,gain", ROPE)
@pytest.mark.parametrize("place", ["new", "inplace", "strided"])
def test_rope(L, gpu, n, h, d, first, rot, inter, inv, dtype, gain, place):
    rng = np.random.default_rng(n + h + d)
    x = torch.from_numpy(rng.standard_normal((n, h, d)).astype(np.float32)).to(dtype)
    pos = rng.integers(0, 200000, n)
    pos[0] = 0
    if n > 2:
        pos[1], pos[2] = 2 ** 31 - 1, -5
    freqs = 10000.0 ** (-np.arange(rot // 2) * 2 / rot)
    dev = x.to(gpu)
    out = None
    if place == "inplace":
        out = dev
    elif place == "strided":                  # a column slice of wider rows, in and out, at offsets that break 16 bytes
        dev = torch.full((n, h, d + 13), 7.0, dtype=dtype, device=gpu)[..., 5:5 + d].copy_(dev)
        out = torch.full((n, h + 1, d + 3), 9.0, dtype=dtype, device=gpu)
        wide, out = out, out[:, :h, 1:1 + d]
    got = L.rope_rotate(dev, torch.from_numpy(pos.astype(np.int32)).to(gpu), torch.from_numpy(freqs).to(gpu), first=first,
                        interleaved=inter, inverse=inv, gain=gain, out=out)
    torch.cuda.synchronize()
    assert out is None or got is out
    x64 = x.double().numpy()
    ref = paged.rope_rotate(x64, pos, freqs, first, inter, inv, gain)
    err = np.abs(got.double().cpu().numpy() - ref)
    tol = _rope_tol(x64, ref, pos, freqs, first, rot, inter, gain, dtype == torch.bfloat16)
    assert (err <= tol).all(), f"{(err - tol).max()} over at {np.unravel_index((err - tol).argmax(), err.shape)}"
    if place == "strided":
        keep = torch.ones_like(wide, dtype=torch.bool)
        keep[:, :h, 1:1 + d] = False
        assert (wide[keep] == 9).all()


def test_rope_four_dimensional_queries(L, gpu):
    """[batch, s_q, heads, d], as the decode takes them."""
    rng = np.random.default_rng(1)
    x = torch.from_numpy(rng.standard_normal((6, 2, 16, 64)).astype(np.float32)).bfloat16()
    pos = rng.integers(0, 5000, 12).astype(np.int32)
    freqs, gain = L.rope_frequencies(64, factor=8.0, device=gpu)
    got = L.rope_rotate(x.to(gpu), torch.from_numpy(pos).to(gpu), freqs, gain=gain)
    flat = L.rope_rotate(x.view(12, 16, 64).to(gpu), torch.from_numpy(pos).to(gpu), freqs, gain=gain)
    assert got.shape == x.shape and torch.equal(got.view(12, 16, 64), flat)


@pytest.mark.parametrize("inter", [False, True])
def test_rope_inverse_is_the_gradient(L, gpu, inter):
    """The map is linear: (f(x + t e) - f(x - t e)) / 2t . g equals (inverse g) . e for any t; fp32, 24 + 24 columns."""
    rng = np.random.default_rng(2)
    n, h, d, first = 4, 3, 64, 8
    x, e, g = (torch.from_numpy(rng.standard_normal((n, h, d)).astype(np.float32)).to(gpu) for _ in range(3))
    pos = torch.tensor([0, 3, 1000, 70000], dtype=torch.int32, device=gpu)
    freqs, gain = L.rope_frequencies(48, factor=4.0, device=gpu)
    f = lambda v: L.rope_rotate(v, pos, freqs, first=first, interleaved=inter, gain=gain).double()  # noqa: E731
    slope = ((f(x + e) - f(x - e)) / 2 * g.double()).sum((1, 2))
    dx = L.rope_rotate(g, pos, freqs, first=first, interleaved=inter, inverse=True, gain=gain)
    want = (dx.double() * e.double()).sum((1, 2))
    # each product is off by at most 2^-20 of magnitudes below 25 (|g| |f|, gain 1.14), 192 of them a token
    assert (slope - want).abs().max().item() <= 192 * 25 * 2.0 ** -20


def test_rope_no_tokens(L, gpu):
    x = torch.zeros((0, 4, 64), dtype=torch.bfloat16, device=gpu)
    freqs, _ = L.rope_frequencies(64, device=gpu)
    assert L.rope_rotate(x, torch.zeros(0, dtype=torch.int32, device=gpu), freqs).shape == x.shape


# ----------------------------------------------------------------------------------------- append

def _append_case(rng, r, dr, news, ctxs, page, std=1.0):
    lens = [n + c for n, c in zip(news, ctxs)]
    n = sum(news)
    x = torch.from_numpy((rng.standard_normal((n, r + dr)) * std).astype(np.float32)).bfloat16()
    need = [-(-v // page) for v in lens]
    order = rng.permutation(sum(need) + 2)
    table = np.full((len(lens), max(1, max(need))), -1, dtype=np.int32)
    at = 0
    for b, v in enumerate(need):
        table[b, :v] = order[at:at + v]
        at += v
    return x, lens, table, sum(need) + 2


APPEND = [
    # r, d_rope, new rows of each request, tokens before them, page size, interleaved, std
    (512, 64, [1], [0], 16, False, 1.0),
    (1024, 64, [2] * 9, [0, 1, 14, 15, 16, 17, 100, 3, 8], 16, False, 1 / 14),
    (256, 64, [0, 5, 0, 0, 33, 1, 0], [3, 0, 0, 9, 2, 40, 1], 7, True, 1.0),
    (32, 8, [70, 1], [0, 5], 1, True, 1e-20),
    (640, 16, [3, 200], [1, 1], 100, False, 1e15),
    (128, 0, [4, 4], [0, 0], 3, False, 1.0),
    (96, 160, [40], [2], 48, False, 1.0),
]


@pytest.mark.parametrize("r,dr,news,ctxs,page,inter,std", APPEND)
def test_append(L, gpu, r, dr, news, ctxs, page, inter, std):
    rng = np.random.default_rng(r + dr + len(news))
    x, lens, table, pages = _append_case(rng, r, dr, news, ctxs, page, std)
    n = sum(news)
    x[0, :32] = 0                                                  # a block of zeros
    x[n // 2, :r] *= torch.from_numpy(rng.choice([1.0, 0.0, 2.0 ** -6], r)).bfloat16()
    x[n - 1, :8] = torch.tensor([7, 0.5, 1.5, 2.5, -0.5, -1.5, 3.5, -7]).bfloat16() * 2.0 ** -3   # ties
    x[n - 1, 8:32] = 0
    rb = L.int4_cache_row_bytes(r, dr)
    pool = torch.full((pages, page, rb + 16), 0x5A, dtype=torch.uint8, device=gpu)   # wider rows: the rest stays
    held = torch.full((n + 2, r + dr), 3.0, dtype=torch.bfloat16, device=gpu)
    rows = torch.full((n + 2, r + dr), 5.0, dtype=torch.bfloat16, device=gpu)        # two rows behind the last request
    rows[:n] = x.to(gpu)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(news)]).astype(np.int32)).to(gpu)
    freqs, gain = L.rope_frequencies(dr, factor=4.0, device=gpu) if dr else (None, 1.0)
    L.paged_append_int4(rows, pool, r, torch.from_numpy(table).to(gpu), torch.tensor(lens, dtype=torch.int32, device=gpu),
                        cu_new=cu, freqs=freqs, gain=gain, interleaved=inter, rows_out=held)
    torch.cuda.synchronize()
    assert L.check_device() == 0
    got = pool.cpu().numpy()
    pos = np.concatenate([np.arange(v - k, v) for v, k in zip(lens, news)]).astype(int)
    req = np.repeat(np.arange(len(news)), news)
    place = [(int(table[b, p // page]), int(p % page)) for b, p in zip(req, pos)]
    mine = np.stack([got[a] for a in place])
    codes, scales = paged.quantize_rows(x[:, :r])
    np.testing.assert_array_equal(paged.unpack_codes(mine[:, :r // 2]), codes)
    sc = torch.from_numpy(mine[:, r // 2:r // 2 + r // 16].copy()).view(torch.bfloat16).double().numpy()
    np.testing.assert_array_equal(sc, scales)
    assert (mine[:, r // 2 + r // 16:rb - 2 * dr] == 0).all() and (mine[:, rb:] == 0x5A).all()
    np.testing.assert_array_equal(held[:n, :r].double().cpu().numpy(), codes * np.repeat(scales, 32, axis=1))
    if dr:
        key = torch.from_numpy(mine[:, rb - 2 * dr:rb].copy()).view(torch.bfloat16)
        assert torch.equal(key, held[:n, r:].cpu())
        x64 = x[:, None, r:].double().numpy()
        ref = paged.rope_rotate(x64, pos, freqs.cpu().numpy(), 0, inter, False, gain)
        tol = _rope_tol(x64, ref, pos, freqs.cpu().numpy(), 0, dr, inter, gain, True)
        assert (np.abs(key.double().numpy()[:, None] - ref) <= tol).all()
    rest = np.ones(got.shape[:2], dtype=bool)
    for a in place:
        rest[a] = False
    assert (got[rest] == 0x5A).all(), "a slot that no new token has was written"
    assert (held[n:] == 3).all(), "a row behind the last request was written"


def test_append_uniform_without_rotation_and_in_place(L, gpu):
    """cu_new=None: n / batch rows each; freqs=None: the key as it comes; rows_out = new_rows; an idle slot and a request
    with fewer tokens than new rows skip the rows that have no place."""
    rng = np.random.default_rng(11)
    r, page, lens = 256, 4, [6, 0, 1, 9]
    x = torch.from_numpy(rng.standard_normal((8, r + 64)).astype(np.float32)).bfloat16()
    table = torch.arange(12, dtype=torch.int32).view(4, 3).to(gpu)
    pool = torch.zeros((12, page, 272), dtype=torch.uint8, device=gpu)
    rows = x.to(gpu)
    L.paged_append_int4(rows, pool, r, table, torch.tensor(lens, dtype=torch.int32, device=gpu), rows_out=rows)
    torch.cuda.synchronize()
    assert L.check_device() == 0
    codes, scales = paged.quantize_rows(x[:, :r])
    want = codes * np.repeat(scales, 32, axis=1)
    written = {0: (0, 4), 1: (0, 5), 5: (2, 0), 6: (3, 7), 7: (3, 8)}     # row -> request, token
    got, back = pool.cpu().numpy(), rows.cpu()
    seen = np.zeros((12, page), dtype=bool)
    for w in range(8):
        if w in written:
            b, t = written[w]
            row = got[3 * b + t // page, t % page]
            seen[3 * b + t // page, t % page] = True
            np.testing.assert_array_equal(paged.unpack_codes(row[None, :r // 2])[0], codes[w])
            np.testing.assert_array_equal(back[w, :r].double().numpy(), want[w])
            assert (row[-128:].view(np.uint16) == bits(x[w, r:])).all()
        else:
            assert torch.equal(back[w], x[w])
    assert (got[~seen] == 0).all()


@pytest.mark.parametrize("bad", [-1, 5, 1 << 30, -(1 << 31)])
def test_append_bad_page_is_recorded_and_skipped(L, gpu, bad):
    pool = torch.zeros((5, 2, 272), dtype=torch.uint8, device=gpu)
    rows = torch.ones((4, 320), dtype=torch.bfloat16, device=gpu)
    table = torch.tensor([[0, bad], [3, 4]], dtype=torch.int32, device=gpu)
    L.paged_append_int4(rows, pool, 256, table, torch.tensor([3, 5], dtype=torch.int32, device=gpu))  # 5 tokens: past the table
    torch.cuda.synchronize()
    assert L.check_device(clear=True) == L.SITE_BAD_ROW
    full = (pool.cpu() != 0).any(-1)
    # request 0: token 1 lands on page 0, token 2 has no page; request 1: token 3 on page 4, token 4 is past the table
    assert full.nonzero().tolist() == [[0, 1], [4, 1]]


# ----------------------------------------------------------------------------------------- decode

DECODE = [
    # d, groups, heads, s_q, lengths, page
    (128, 8, 128, 1, [37], 16),
    (128, 8, 128, 2, [1, 2, 3, 127, 128, 129, 255, 256, 257], 16),
    (128, 8, 128, 2, [0, 0, 300, 0, 1, 0], 48),
    (128, 4, 32, 1, [0, 5, 1000, 64, 129, 640], 32),
    (128, 2, 128, 1, [700, 130], 100),                            # 64 rows a group
    (128, 2, 128, 2, [257, 1, 0, 513], 64),                       # 128 rows a group
    (128, 1, 1, 1, [1, 500], 3),                                  # one head
    (128, 1, 3, 2, [129, 40], 1),                                 # pages of one token
    (128, 1, 40, 2, [300], 512),                                  # a page longer than the request
    (256, 2, 128, 1, [300, 129, 1, 0, 4000], 64),                 # GLA-2
    (256, 2, 128, 2, [255, 65], 64),
    (256, 4, 20, 1, [400, 3], 48),
    (256, 1, 128, 2, [130, 1], 16),                               # 256 rows a group
    (512, 1, 128, 1, [1, 130, 64, 0, 500], 64),                   # MLA absorbed
    (512, 1, 128, 2, [129, 1, 300], 16),
    (512, 2, 12, 2, [200, 2], 33),
    (128, 3, 9, 1, [200, 333], 16),                               # three groups
    (128, 5, 60, 2, [2100, 17], 16),
]


def _decode(L, gpu, q, qr, pool, G, table, lens, scale, **kw):
    return L.paged_decode_int4(q.to(gpu), qr.to(gpu), torch.from_numpy(pool).to(gpu), G, torch.from_numpy(table).to(gpu),
                               torch.tensor(lens, dtype=torch.int32, device=gpu), scale, **kw)


@pytest.mark.parametrize("d,G,H,s_q,lens,page", DECODE)
def test_decode(L, gpu, d, G, H, s_q, lens, page):
    rng = np.random.default_rng(d + G + H + s_q + sum(lens))
    pool, table = make_pool(rng, lens, G, d, page)
    q, qr = queries(rng, len(lens), s_q, H, d)
    scale = 1 / math.sqrt(d + D_ROPE)
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device=gpu)
    lse = torch.full(q.shape[:-1], float("nan"), device=gpu)
    _decode(L, gpu, q, qr, pool, G, table, lens, scale, out=out, lse=lse)
    torch.cuda.synchronize()
    assert L.check_device() == 0
    ref = paged.paged_decode(q, qr, pool, G, table, lens, scale)
    print(check_decode(out, lse, ref, d, max(lens), f"d={d} G={G} H={H}"))


@pytest.mark.parametrize("d,G,H,s_q", [(128, 8, 64, 2), (256, 2, 64, 1), (512, 1, 64, 1)])
@pytest.mark.parametrize("kind", ["wide", "equal", "rising", "falling", "late_peak"])
def test_decode_score_ranges(L, gpu, d, G, H, s_q, kind):
    """Scores that spread over hundreds of nats, are all equal, rise or fall along the keys, or peak at the last one: the
    running maximum has to move, or must not."""
    rng = np.random.default_rng(len(kind) + d)
    lens, page = [700, 385], 32
    pool, table = make_pool(rng, lens, G, d, page)
    q, qr = queries(rng, len(lens), s_q, H, d, std=0.0 if kind == "equal" else 20.0 if kind == "wide" else 0.25)
    r = G * d
    if kind in ("rising", "falling", "late_peak"):
        qr[..., 0] = 8.0
        for b, n in enumerate(lens):
            for t in range(n):
                f = t / n if kind == "rising" else -t / n if kind == "falling" else float(t == n - 1)
                key = torch.tensor([f * 400]).bfloat16()
                pool[table[b, t // page], t % page, paged.row_bytes(r, 64) - 128:][:2] = key.view(torch.uint8).numpy()
    scale = 1 / math.sqrt(d + D_ROPE)
    out, lse = _decode(L, gpu, q, qr, pool, G, table, lens, scale)
    torch.cuda.synchronize()
    assert L.check_device() == 0
    check_decode(out, lse, paged.paged_decode(q, qr, pool, G, table, lens, scale), d, max(lens), kind)


def test_decode_pool_and_table_views(L, gpu):
    """A pool that is a view of wider rows and of every second page, a table that is a slice of a wider one."""
    rng = np.random.default_rng(21)
    d, G, H, lens, page = 128, 4, 16, [90, 300, 17], 16
    pool, table = make_pool(rng, lens, G, d, page)
    q, qr = queries(rng, 3, 1, H, d)
    a = _decode(L, gpu, q, qr, pool, G, table, lens, 0.07)
    big = torch.full((2 * pool.shape[0], page + 1, pool.shape[2] + 48), 0xFF, dtype=torch.uint8, device=gpu)
    view = big[1::2, 1:, 16:16 + pool.shape[2]]
    view.copy_(torch.from_numpy(pool))
    wide = torch.full((3, table.shape[1] + 5), 1 << 20, dtype=torch.int32, device=gpu)
    wide[:, :table.shape[1]] = torch.from_numpy(table).to(gpu)
    b = L.paged_decode_int4(q.to(gpu), qr.to(gpu), view, G, wide, torch.tensor(lens, dtype=torch.int32, device=gpu), 0.07)
    torch.cuda.synchronize()
    assert L.check_device() == 0
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_decode_ignores_rows_behind_the_end(L, gpu):
    """Slots behind a request's last token, unused pages and unused table entries change nothing, bit for bit."""
    d, G, H, lens, page = 256, 2, 32, [130, 1, 77], 48
    got = []
    for junk in (0x00, 0xFF, 0x7F):
        rng = np.random.default_rng(22)
        pool, table = make_pool(rng, lens, G, d, page, junk=junk)
        table[table < 0] = junk << 16
        q, qr = queries(rng, 3, 2, H, d)
        got.append(_decode(L, gpu, q, qr, pool, G, table, lens, 0.05))
    torch.cuda.synchronize()
    assert L.check_device() == 0
    for o, l in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(l, got[0][1])


def test_decode_missing_page_is_recorded_and_others_stand(L, gpu):
    """A token without a page counts as a row of zeros; the other requests' results are untouched."""
    rng = np.random.default_rng(23)
    d, G, H, lens, page = 128, 2, 8, [200, 150, 90], 32
    pool, table = make_pool(rng, lens, G, d, page)
    q, qr = queries(rng, 3, 1, H, d)
    want = _decode(L, gpu, q, qr, pool, G, table, lens, 0.07)
    torch.cuda.synchronize()
    assert L.check_device() == 0
    broken = table.copy()
    broken[1, 2] = pool.shape[0]
    got = _decode(L, gpu, q, qr, pool, G, broken, lens, 0.07)
    torch.cuda.synchronize()
    assert L.check_device(clear=True) == L.SITE_BAD_ROW
    for b in (0, 2):
        assert torch.equal(got[0][b], want[0][b]) and torch.equal(got[1][b], want[1][b])
    zeroed = pool.copy()
    zeroed[table[1, 2]] = 0
    zeroed[table[1, 2], :, :G * d // 2] = 0x88
    check_decode(got[0], got[1], paged.paged_decode(q, qr, zeroed, G, table, lens, 0.07), d, 200)
    # a request longer than its table: the same
    L.paged_decode_int4(q.to(gpu), qr.to(gpu), torch.from_numpy(pool).to(gpu), G, torch.from_numpy(table[:, :2].copy()).to(gpu),
                        torch.tensor(lens, dtype=torch.int32, device=gpu), 0.07)
    torch.cuda.synchronize()
    assert L.check_device(clear=True) == L.SITE_BAD_ROW


def test_decode_pages_shared_by_requests(L, gpu):
    """Two requests with the same prefix pages give what two copies of them give."""
    rng = np.random.default_rng(24)
    d, G, H, page = 128, 4, 32, 16
    pool, table = make_pool(rng, [64, 64], G, d, page)
    q, qr = queries(rng, 2, 1, H, d)
    shared = table.copy()
    shared[1] = shared[0]
    copy = pool.copy()
    copy[table[1]] = pool[table[0]]
    a = _decode(L, gpu, q, qr, pool, G, shared, [64, 50], 0.07)
    b = _decode(L, gpu, q, qr, copy, G, table, [64, 50], 0.07)
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# Pages against the copies: runs of 8 .. 128 rows within a page, or single rows; every width of group, few rows and many.
@pytest.mark.parametrize("d,G,H,s_q,lens,page", [
    (128, 8, 128, 1, [200, 9], 8), (128, 4, 128, 1, [130, 500], 24), (128, 7, 14, 1, [385], 40), (128, 2, 128, 1, [300], 96),
    (128, 1, 16, 1, [129, 640], 128), (128, 3, 60, 2, [700, 256], 256), (128, 2, 24, 1, [1500], 1000), (128, 5, 5, 1, [300], 7),
    (256, 2, 16, 1, [200, 9], 8), (256, 3, 60, 2, [130, 500], 24), (256, 4, 256, 1, [385], 40), (256, 1, 30, 1, [300, 77], 1),
    (256, 2, 128, 1, [700, 256], 256), (256, 1, 8, 2, [260], 9), (512, 1, 20, 1, [300, 40], 8), (512, 2, 60, 2, [131], 5)])
def test_decode_page_sizes(L, gpu, d, G, H, s_q, lens, page):
    rng = np.random.default_rng(31)
    pool, table = make_pool(rng, lens, G, d, page)
    q, qr = queries(rng, len(lens), s_q, H, d)
    out, lse = _decode(L, gpu, q, qr, pool, G, table, lens, 1 / math.sqrt(d + D_ROPE))
    torch.cuda.synchronize()
    assert L.check_device() == 0
    check_decode(out, lse, paged.paged_decode(q, qr, pool, G, table, lens, 1 / math.sqrt(d + D_ROPE)), d, max(lens))


@pytest.mark.parametrize("d,G,H,page", [(128, 2, 8, 8), (128, 2, 60, 3), (256, 2, 8, 16), (256, 2, 128, 5), (512, 1, 16, 16)])
def test_decode_missing_pages_count_as_zero_rows(L, gpu, d, G, H, page):
    rng = np.random.default_rng(32)
    lens = [300, 140]
    pool, table = make_pool(rng, lens, G, d, page)
    q, qr = queries(rng, 2, 1, H, d)
    broken, zeroed = table.copy(), pool.copy()
    for k in (0, 1, 4, 140 // page):
        broken[0, k] = -7 if k % 2 else pool.shape[0] + k
        zeroed[table[0, k]] = 0
        zeroed[table[0, k], :, :G * d // 2] = 0x88
    out, lse = _decode(L, gpu, q, qr, pool, G, broken, lens, 0.05)
    torch.cuda.synchronize()
    assert L.check_device(clear=True) == L.SITE_BAD_ROW
    check_decode(out, lse, paged.paged_decode(q, qr, zeroed, G, table, lens, 0.05), d, 300)


@pytest.mark.parametrize("d,G,H", [(128, 2, 8), (256, 2, 40), (512, 1, 70)])
def test_pool_with_rows_of_pages_side_by_side(L, gpu, d, G, H):
    """Slot s of all pages side by side (rows further apart than pages): append and decode give what whole pages give."""
    rng = np.random.default_rng(33)
    lens, page, r = [90, 300], 16, G * d
    pool, table = make_pool(rng, lens, G, d, page)
    q, qr = queries(rng, 2, 1, H, d)
    rows = torch.from_numpy(rng.standard_normal((6, r + 64)).astype(np.float32)).bfloat16().to(gpu)
    whole = torch.from_numpy(pool).to(gpu)
    side = torch.empty((page,) + (pool.shape[0], pool.shape[2]), dtype=torch.uint8, device=gpu).transpose(0, 1)
    side.copy_(whole)
    assert side.stride(0) < side.stride(1)
    t, n = torch.from_numpy(table).to(gpu), torch.tensor(lens, dtype=torch.int32, device=gpu)
    got = []
    for place in (whole, side):
        L.paged_append_int4(rows, place, r, t, n)
        got.append(L.paged_decode_int4(q.to(gpu), qr.to(gpu), place, G, t, n, 0.06))
    torch.cuda.synchronize()
    assert L.check_device() == 0
    assert torch.equal(whole, side)
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("d,G", [(128, 8), (256, 4), (512, 2)])
def test_pool_past_32_bit_offsets(L, gpu, d, G):
    """Pages more than 2^32 bytes into the pool: append and decode give what a small pool gives."""
    rng = np.random.default_rng(34)
    lens, page, r, H = [150, 33], 64, G * d, 8 * G
    pool, table = make_pool(rng, lens, G, d, page)
    q, qr = queries(rng, 2, 1, H, d)
    rows = torch.from_numpy(rng.standard_normal((4, r + 64)).astype(np.float32)).bfloat16().to(gpu)
    small, n = torch.from_numpy(pool).to(gpu), torch.tensor(lens, dtype=torch.int32, device=gpu)
    first = -(-((1 << 32) + 12345) // (page * pool.shape[2]))
    large = torch.empty((first + pool.shape[0], page, pool.shape[2]), dtype=torch.uint8, device=gpu)
    large[first:].copy_(small)
    got = []
    for place, t in ((small, table), (large, np.where(table >= 0, table + first, table))):
        t = torch.from_numpy(t.astype(np.int32)).to(gpu)
        L.paged_append_int4(rows, place, r, t, n)
        got.append(L.paged_decode_int4(q.to(gpu), qr.to(gpu), place, G, t, n, 0.06))
    torch.cuda.synchronize()
    assert L.check_device() == 0
    assert torch.equal(large[first:], small)
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def test_two_captured_graphs_replayed_in_turn(L, gpu):
    """Two captured decodes, each with outputs and a workspace of its capture's own: replays in any order, and on two
    streams at once, give what plain calls give."""
    rng = np.random.default_rng(35)
    cases = []
    for d, G, H, lens, page in [(128, 4, 64, [2000, 70], 32), (256, 2, 64, [900, 1, 300], 64)]:
        pool, table = make_pool(rng, lens, G, d, page)
        q, qr = queries(rng, len(lens), 1, H, d)
        args = (q.to(gpu), qr.to(gpu), torch.from_numpy(pool).to(gpu), G, torch.from_numpy(table).to(gpu),
                torch.tensor(lens, dtype=torch.int32, device=gpu), 0.06)
        want = L.paged_decode_int4(*args)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = L.paged_decode_int4(*args)
        cases.append((graph, got, want, args))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for order in ((0, 1), (1, 0), (0, 0), (1, 1)):
        for _, got, _, _ in cases:
            got[0].fill_(float("nan"))
        torch.cuda.synchronize()
        for s, k in zip((s1, s2) if order[0] != order[1] else (s1, s1), order):
            with torch.cuda.stream(s):
                cases[k][0].replay()
        torch.cuda.synchronize()
        for k in set(order):
            _, got, want, _ = cases[k]
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert L.check_device() == 0


def test_decode_runs_repeat_bit_for_bit_and_on_two_streams(L, gpu):
    rng = np.random.default_rng(25)
    d, G, H, lens, page = 128, 8, 128, [3000, 10, 900], 64
    pool, table = make_pool(rng, lens, G, d, page)
    q, qr = queries(rng, 3, 2, H, d)
    args = (q.to(gpu), qr.to(gpu), torch.from_numpy(pool).to(gpu), G, torch.from_numpy(table).to(gpu),
            torch.tensor(lens, dtype=torch.int32, device=gpu), 0.07)
    want = L.paged_decode_int4(*args)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(5):
        got.append(L.paged_decode_int4(*args, stream=s1))
        with torch.cuda.stream(s2):
            got.append(L.paged_decode_int4(*args))
    torch.cuda.synchronize()
    for o, l in got:
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])


def test_step_captured_and_replayed(L, gpu):
    """Rotate the queries, append the step's rows and decode, captured once and replayed with the lengths moved on: each
    replay equals the same calls made one by one, and the oracle over the pool it left."""
    rng = np.random.default_rng(26)
    d, G, H, s_q, page, B = 128, 4, 32, 2, 16, 3
    r, lens0 = G * d, [40, 130, 0]
    pool0, _ = make_pool(rng, [200] * B, G, d, page, junk=0)
    pages = 13
    table = torch.arange(B * pages, dtype=torch.int32).view(B, pages).to(gpu)
    freqs, gain = L.rope_frequencies(64, factor=2.0, device=gpu)
    scale = 1 / math.sqrt(d + D_ROPE)
    steps = [(queries(rng, B, s_q, H, d),
              torch.from_numpy(rng.standard_normal((B * s_q, r + 64)).astype(np.float32)).bfloat16()) for _ in range(3)]

    def state():
        return {"pool": torch.from_numpy(pool0.copy()).to(gpu), "lens": torch.tensor(lens0, dtype=torch.int32, device=gpu),
                "pos": torch.zeros(B * s_q, dtype=torch.int32, device=gpu),
                "q": torch.zeros((B, s_q, H, d), dtype=torch.bfloat16, device=gpu),
                "qr": torch.zeros((B, s_q, H, 64), dtype=torch.bfloat16, device=gpu),
                "rows": torch.zeros((B * s_q, r + 64), dtype=torch.bfloat16, device=gpu)}

    def load(s, step, lens):
        (q, qr), rows = step
        s["q"].copy_(q.to(gpu))
        s["qr"].copy_(qr.to(gpu))
        s["rows"].copy_(rows.to(gpu))
        s["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        s["pos"].copy_((torch.tensor(lens)[:, None] - s_q + torch.arange(s_q)).clamp(min=0).reshape(-1).int())

    def call(s, out, lse, ws):
        turned = L.rope_rotate(s["qr"], s["pos"], freqs, gain=gain)
        L.paged_append_int4(s["rows"], s["pool"], r, table, s["lens"], freqs=freqs, gain=gain)
        L.paged_decode_int4(s["q"], turned, s["pool"], G, table, s["lens"], scale, out=out, lse=lse, workspace=ws)
        return turned

    sms = torch.cuda.get_device_properties(gpu).multi_processor_count
    new = lambda: (torch.empty((B, s_q, H, d), dtype=torch.bfloat16, device=gpu), torch.empty((B, s_q, H), device=gpu),  # noqa: E731
                   torch.empty(L.paged_decode_workspace_size(B, s_q, H, G, d, sms), dtype=torch.uint8, device=gpu))
    a, b = state(), state()
    oa, ob = new(), new()
    load(a, steps[0], [2, 2, 2])
    call(a, *oa)                                    # warm up before the capture
    torch.cuda.synchronize()
    a["pool"].copy_(torch.from_numpy(pool0))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(a, *oa)
    lens = list(lens0)
    for k, step in enumerate(steps):
        lens = [n + s_q if not (k == 0 and b_ == 2) else 0 for b_, n in enumerate(lens)]   # the third request joins later
        load(a, step, lens)
        load(b, step, lens)
        graph.replay()
        turned = call(b, *ob)
        torch.cuda.synchronize()
        assert L.check_device() == 0
        assert torch.equal(oa[0], ob[0]) and torch.equal(oa[1], ob[1]) and torch.equal(a["pool"], b["pool"])
        ref = paged.paged_decode(step[0][0], turned.cpu(), a["pool"].cpu().numpy(), G, table.cpu().numpy(), lens, scale)
        check_decode(oa[0], oa[1], ref, d, max(lens), f"step {k}")


def test_binding_refusals_on_the_gpu(L, gpu):
    pool = torch.zeros((4, 16, 704), dtype=torch.uint8, device=gpu)
    table, lens = torch.zeros((2, 3), dtype=torch.int32, device=gpu), torch.ones(2, dtype=torch.int32, device=gpu)
    q, qr = torch.zeros((2, 1, 128, 128), dtype=torch.bfloat16, device=gpu), torch.zeros((2, 1, 128, 64), dtype=torch.bfloat16, device=gpu)
    ok = lambda **kw: L.paged_decode_int4(*[kw.get(k, v) for k, v in dict(q=q, qr=qr, pool=pool, g=8, table=table, lens=lens, scale=0.07).items()])  # noqa: E731
    ok()
    for kw, e in [(dict(lens=lens.cpu()), ValueError), (dict(table=table.cpu()), ValueError), (dict(pool=pool[..., :600]), ValueError),
                  (dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)[:, :, ::2], qr=qr[:, :, ::2]), ValueError),
                  (dict(table=table.T.contiguous().T), ValueError), (dict(lens=lens[:1]), ValueError),
                  (dict(qr=qr[..., :32].contiguous()), (ValueError, L.LkvError)), (dict(scale=-1.0), L.LkvError)]:
        with pytest.raises(e):
            ok(**kw)
    with pytest.raises(L.LkvError) as err:
        L.paged_decode_int4(q, qr, pool, 8, table, lens, 0.07, workspace=torch.empty(16, dtype=torch.uint8, device=gpu))
    assert err.value.status == L.ERR_WORKSPACE
    rows = torch.zeros((4, 1088), dtype=torch.bfloat16, device=gpu)
    for kw in [dict(cu_new=torch.zeros(2, dtype=torch.int32, device=gpu)), dict(freqs=torch.zeros(16, dtype=torch.float64, device=gpu)),
               dict(rows_out=rows[:2])]:
        with pytest.raises(ValueError):
            L.paged_append_int4(rows, pool, 1024, table, lens, **kw)
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16, device=gpu)
    f = torch.zeros(32, dtype=torch.float64, device=gpu)
    for a in [(x[0], torch.zeros(2, dtype=torch.int32, device=gpu)), (x, torch.zeros(5, dtype=torch.int32, device=gpu)),
              (x.transpose(1, 2), torch.zeros(4, dtype=torch.int32, device=gpu))]:
        with pytest.raises(ValueError):
            L.rope_rotate(*a, f)
    with pytest.raises(L.LkvError):
        L.rope_rotate(x, torch.zeros(4, dtype=torch.int32, device=gpu), f, first=2)
    torch.cuda.synchronize()
    assert L.check_device() == 0
