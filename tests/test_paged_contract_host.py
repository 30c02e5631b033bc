"""What the documentation of the rotary and paged entry points promises beside the results, without a GPU."""
import math

import torch


def test_interpolation_of_the_positions_has_gain_one(lkv_built):
    """beta_fast = inf divides every frequency, which is the plain map at positions divided by factor: no gain."""
    f, gain = lkv_built.rope_frequencies(64, factor=4.0, beta_fast=math.inf)
    plain, _ = lkv_built.rope_frequencies(64)
    assert torch.allclose(f, plain / 4, rtol=1e-15) and gain == 1.0
    assert lkv_built.rope_frequencies(64, factor=4.0)[1] == 1.0 + 0.1 * math.log(4.0)


def test_whole_number_arrays_off_their_alignment_are_refused(lkv_built):
    """The kernels load positions, lengths and tables as 32-bit words."""
    from test_paged_host import GOOD, _append, _decode, _rope
    L = lkv_built
    assert _rope(L, pos=GOOD + 2) == L.ERR_INVALID_ARG
    for kw in [dict(table=GOOD + 1), dict(lens=GOOD + 2), dict(cu=GOOD + 3)]:
        assert _append(L, **kw) == L.ERR_INVALID_ARG, kw
    for kw in [dict(table=GOOD + 2), dict(lens=GOOD + 3)]:
        assert _decode(L, **kw) == L.ERR_INVALID_ARG, kw


def test_rope_refuses_a_result_whose_rows_overlap(lkv_built):
    """Two rows that share an element would be written by two threads, and in place read by one after the other's write."""
    from test_paged_host import GOOD, _rope
    L = lkv_built
    two = dict(x=GOOD, out=1 << 24, n=4, heads=16, d=64)
    for kw in [dict(o_ts=0), dict(o_hs=0), dict(o_ts=63), dict(o_hs=32, o_ts=1024), dict(o_ts=-1, o_hs=-64), dict(o_ts=512, o_hs=64),
               dict(o_ts=64, o_hs=128), dict(n=100, o_ts=64, o_hs=6399), dict(n=2, heads=12, o_ts=700, o_hs=64),
               dict(n=3, o_ts=160, o_hs=104), dict(out=GOOD, x_ts=0, o_ts=0), dict(out=GOOD, x_hs=0, o_hs=0)]:
        assert _rope(L, **{**two, **kw}) == L.ERR_INVALID_ARG, kw


def _overlap(ts, n, hs, heads, d):
    rows = sorted(t * ts + h * hs for t in range(n) for h in range(heads))
    return any(b - a < d for a, b in zip(rows, rows[1:]))


def test_rope_takes_every_layout_whose_rows_lie_apart(lkv_built):
    """By brute force over small layouts, heads within tokens, tokens within heads and interleaved ones among them.  Without a
    GPU a call that passes the checks ends in the launch's error; on one nothing is called."""
    import itertools
    import pytest
    from test_paged_host import GOOD, _rope
    L = lkv_built
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")
    seen = [0, 0]
    for n, heads, d in [(1, 1, 4), (1, 5, 4), (5, 1, 4), (2, 3, 4), (4, 3, 2), (3, 7, 4)]:
        for ts, hs in itertools.product(range(0, 34, 1), repeat=2):
            over = _overlap(ts, n, hs, heads, d)
            seen[over] += 1
            got = _rope(L, x=GOOD, out=1 << 24, n=n, heads=heads, d=d, rot=2, o_ts=ts, o_hs=-hs if ts % 3 == 0 else hs)
            assert got == (L.ERR_INVALID_ARG if over else L.ERR_CUDA), (n, heads, d, ts, hs)
    assert min(seen) > 500
