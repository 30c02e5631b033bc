"""Rows with NaN and infinities through the 4-bit append and the decode: what is no number is held as NaN and reaches the
results of its own request, and of no other."""
import math

import numpy as np
import pytest
import torch

from oracle import paged
from paged_large_util import make_large, make_queries
from paged_util import D_ROPE

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L(gpu):
    import latent_kv_cache_split_b200 as lib
    lib.check_device(clear=True)
    return lib


@pytest.mark.parametrize("r", [32, 512, 1024])
def test_append_holds_a_block_with_what_is_no_number_as_nan(L, gpu, r):
    rng = np.random.default_rng(r)
    n, page = 11, 4
    x = torch.from_numpy(rng.standard_normal((n, r + D_ROPE)).astype(np.float32)).bfloat16()
    bad = [(0, 0, NAN), (1, 31, INF), (2, 17, -INF), (3, r - 1, NAN), (4, r // 2, -NAN), (5, r - 32, INF), (5, r - 31, NAN)]
    blocks = np.zeros((n, r // 32), dtype=bool)
    for t, c, v in bad:
        x[t, c] = v
        blocks[t, c // 32] = True
    x[6, r], x[7, r + 63] = NAN, INF              # the RoPE key is carried as it is
    pool = torch.zeros((4, page, L.int4_cache_row_bytes(r, D_ROPE)), dtype=torch.uint8, device=gpu)
    held = torch.zeros((n, r + D_ROPE), dtype=torch.bfloat16, device=gpu)
    table = torch.tensor([[2, 0, 3]], dtype=torch.int32, device=gpu)
    L.paged_append_int4(x.to(gpu), pool, r, table, torch.tensor([n], dtype=torch.int32, device=gpu), rows_out=held)
    torch.cuda.synchronize()
    assert L.check_device() == 0
    rows = torch.stack([pool[int(table[0, t // page]), t % page] for t in range(n)])
    codes, scales, key = (f.cpu() for f in L.int4_cache_fields(rows, r, D_ROPE))
    clean = torch.where(torch.from_numpy(np.repeat(blocks, 32, axis=1)), 0.0, x[:, :r].float())
    want_codes, want_scales = paged.quantize_rows(clean)
    want_scales[blocks] = np.nan
    stand = ~np.repeat(blocks, 32, axis=1)
    np.testing.assert_array_equal(paged.unpack_codes(codes.numpy())[stand], want_codes[stand])
    np.testing.assert_array_equal(scales.double().numpy(), want_scales)
    np.testing.assert_array_equal(held[:, :r].double().cpu().numpy(), want_codes * np.repeat(want_scales, 32, axis=1))
    np.testing.assert_array_equal(key.float().numpy(), x[:, r:].float().numpy())


@pytest.mark.parametrize("d,G,H,page", [(128, 2, 16, 16), (128, 2, 64, 16), (128, 4, 200, 4), (256, 2, 16, 5), (256, 2, 128, 64), (512, 1, 40, 16)])
@pytest.mark.parametrize("value", [NAN, INF])
def test_decode_of_such_a_row_is_nan_in_its_request_alone(L, gpu, d, G, H, page, value):
    """The row's group: NaN in every head's lse and results; other groups and requests: the bits of a clean cache."""
    lens, r = [700, 90, 1500], G * d
    pool, table = make_large(lens, G, d, page, d, gpu)
    q, qr = make_queries(3, 1, H, d, H, gpu)
    n = torch.tensor(lens, dtype=torch.int32, device=gpu)
    row = torch.randn((1, r + D_ROPE), device=gpu).to(torch.bfloat16)
    got = []
    for v in (0.5, value):
        row[0, 3] = v                             # group 0
        one = torch.tensor([0, 0, 0, 1], dtype=torch.int32, device=gpu)
        L.paged_append_int4(row, pool, r, table, n, cu_new=one)
        got.append(L.paged_decode_int4(q, qr, pool, G, table, n, 1 / math.sqrt(d + D_ROPE)))
    torch.cuda.synchronize()
    assert L.check_device() == 0
    (clean, clean_lse), (out, lse) = got
    h = H // G
    assert torch.isnan(out[2, :, :h]).all() and torch.isnan(lse[2, :, :h]).all()
    assert torch.equal(out[:2], clean[:2]) and torch.equal(lse[:2], clean_lse[:2])
    assert torch.equal(out[2, :, h:], clean[2, :, h:]) and torch.equal(lse[2, :, h:], clean_lse[2, :, h:])
    assert torch.isfinite(clean).all() and torch.isfinite(clean_lse).all()


@pytest.mark.parametrize("d,G,H,page", [(128, 2, 16, 16), (128, 2, 64, 5), (256, 2, 128, 64), (512, 1, 40, 16)])
def test_the_older_query_loses_the_columns_held_as_nan_alone(L, gpu, d, G, H, page):
    """s_q = 2 and the newest token's row: the older query does not see it, but its value columns meet a weight of 0."""
    lens, r = [400, 257], G * d
    pool, table = make_large(lens, G, d, page, d, gpu)
    q, qr = make_queries(2, 2, H, d, H, gpu)
    n = torch.tensor(lens, dtype=torch.int32, device=gpu)
    row = torch.randn((1, r + D_ROPE), device=gpu).to(torch.bfloat16)
    got = []
    for v in (0.5, NAN):
        row[0, 40] = v                            # columns 32 .. 63 of group 0
        L.paged_append_int4(row, pool, r, table, n, cu_new=torch.tensor([0, 1, 1], dtype=torch.int32, device=gpu))
        got.append(L.paged_decode_int4(q, qr, pool, G, table, n, 0.06))
    torch.cuda.synchronize()
    assert L.check_device() == 0
    (clean, clean_lse), (out, lse) = got
    h = H // G
    assert torch.isnan(out[0, 1, :h]).all() and torch.isnan(lse[0, 1, :h]).all()
    assert torch.equal(lse[0, 0], clean_lse[0, 0]) and torch.isnan(out[0, 0, :h, 32:64]).all()
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[0, 1, :h] = False
    keep[0, 0, :h, 32:64] = False
    assert torch.equal(out[keep], clean[keep]) and torch.isfinite(clean).all()


def test_append_skips_the_rows_of_the_least_length(L, gpu):
    """A length of 0 or less is an idle slot, the least int32 too: its rows have no place and no error is recorded."""
    r, rows = 32, torch.ones((4, 32 + D_ROPE), dtype=torch.bfloat16, device=gpu)
    pool = torch.zeros((2, 1 << 20, 160), dtype=torch.uint8, device=gpu)
    table = torch.tensor([[0] * 4, [1] * 4], dtype=torch.int32, device=gpu)
    for least in (-(1 << 31), -(1 << 31) + 1, -3, 0):
        n = torch.tensor([least, 2], dtype=torch.int32, device=gpu)
        for cu in (None, torch.tensor([0, 2, 4], dtype=torch.int32, device=gpu)):
            L.paged_append_int4(rows, pool, r, table, n, cu_new=cu)
            torch.cuda.synchronize()
            assert L.check_device(clear=True) == 0
    assert (pool[0] == 0).all() and (pool[1, :2] != 0).any() and (pool[1, 2:] == 0).all()
