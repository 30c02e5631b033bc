"""The helpers of the large decode tests, on the CPU: their fp64 decode equals the oracle's, and the inputs whose scores move
between tiles tell a walk that keeps its sums in step with its references from one that does not."""
import math

import numpy as np
import pytest
import torch

from oracle import paged
from paged_large_util import decode64, make_large, make_queries, ragged, tiles
from paged_util import D_ROPE, check_decode


@pytest.mark.parametrize("d,G,H,s_q,page", [(128, 2, 6, 2, 5), (512, 1, 3, 1, 16), (256, 3, 6, 2, 48)])
def test_decode64_equals_the_oracle(d, G, H, s_q, page):
    lens = [0, 1, 7, 130]
    pool, table = make_large(lens, G, d, page, 3, "cpu", key0=lambda b, t: t % 5 * 8)
    q, qr = make_queries(len(lens), s_q, H, d, 4, "cpu")
    got = decode64(q, qr, pool, G, table, lens, 0.07)
    want = paged.paged_decode(q, qr, pool.numpy(), G, table.numpy(), lens, 0.07)
    for a, b in zip(got, want):
        np.testing.assert_allclose(a, b, atol=1e-11, rtol=1e-12)


def test_ragged_lengths_and_their_tiles():
    lens = ragged(50, 400, 1, 3000)
    assert len(lens) == 53 and lens.count(0) == 3 and 1 in lens and max(lens) >= 3000
    assert tiles([0, -2, 1, 128, 129]) == 4


def _walk(s, v, raise_at, fault):
    """Rows' scores s [R, n] (log2 units) and values v [n, d] as the kernel takes them: tiles of 128, two groups in turn, a
    reference a row that all rows raise when one row passes it by raise_at; `fault` leaves a step out."""
    R, n = s.shape
    ref, l, o = [None, None], np.zeros((2, R)), np.zeros((2, R, v.shape[1]))
    rises = 0
    for k, t in enumerate(range(0, n, 128)):
        g, x, y = k % 2, s[:, t:t + 128], v[t:t + 128]
        if ref[g] is None:
            ref[g] = x.max(1)
        elif (x - ref[g][:, None]).max() > raise_at:
            up = np.maximum(x.max(1) - ref[g], 0)
            ref[g] = ref[g] + up
            rises += 1
            if fault != "sums":
                l[g] *= 2.0 ** -up
            if fault != "outputs":
                o[g] *= 2.0 ** -up[:, None]
        w = 2.0 ** (x - ref[g][:, None])
        l[g] += w.sum(1)
        o[g] += w @ y
    top = np.maximum(*ref)
    f = [np.ones(R) if fault == "join" else 2.0 ** (r - top) for r in ref]
    total = f[0] * l[0] + f[1] * l[1]
    return (f[0][:, None] * o[0] + f[1][:, None] * o[1]) / total[:, None], (top + np.log2(total)) * math.log(2), rises


@pytest.mark.parametrize("wave", [(0, 0, 80, 80, 160, 160, 80, 80), (0, 80, 0, 160, 0, 80, 0, 40)])
@pytest.mark.parametrize("fault", [None, "sums", "outputs", "join"])
def test_moving_scores_tell_a_wrong_walk(fault, wave):
    d, H, n = 128, 10, 128 * 9 - 50
    at = torch.tensor(wave)
    pool, table = make_large([n], 1, d, 16, 5, "cpu", key0=lambda b, t: at[t // 128 % len(wave)])
    q, qr = make_queries(1, 1, H, d, 6, "cpu")
    qr[..., 0] = torch.tensor([16.0, 0.0, -16.0, 0.5, -2.0]).repeat(2)
    scale = 1 / math.sqrt(d + D_ROPE)
    ref = decode64(q, qr, pool, 1, table, [n], scale)
    rows = pool[table[0].long()].flatten(0, 1)[:n].numpy()
    sc = torch.from_numpy(rows[:, d // 2:d // 2 + d // 16].copy()).view(torch.bfloat16).double().numpy()
    lat = paged.unpack_codes(rows[:, :d // 2]) * np.repeat(sc, 32, axis=1)
    kpe = torch.from_numpy(rows[:, -2 * D_ROPE:].copy()).view(torch.bfloat16).double().numpy()
    s = scale / math.log(2) * (q[0, 0].double().numpy() @ lat.T + qr[0, 0].double().numpy() @ kpe.T)
    out, lse, rises = _walk(s, lat, 24.0, fault)
    assert rises >= 2
    got = torch.from_numpy(out).bfloat16()[None, None], torch.from_numpy(lse).float()[None, None]
    if fault is None:
        check_decode(*got, ref, d, n)
    else:
        with pytest.raises(AssertionError):
            check_decode(*got, ref, d, n)
