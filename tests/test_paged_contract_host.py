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
