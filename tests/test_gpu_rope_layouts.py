"""rope_rotate over views whose leading dimensions have no common stride: the same results as over their copies."""
import numpy as np
import pytest
import torch

from test_gpu_paged import L  # noqa: F401  (the library's fixture)

pytestmark = pytest.mark.gpu

VIEWS = {
    "tokens cut": lambda x: x[:, 1:-1],
    "heads first": lambda x: x.transpose(1, 2),
    "columns and every second token": lambda x: x[:, ::2, :, 3:],
    "five dimensions": lambda x: x.view(2, 3, 7, 6, 64)[:, :, 2:],
    "no tokens": lambda x: x[:, 3:3],
}


@pytest.mark.parametrize("view", VIEWS)
@pytest.mark.parametrize("place", ["new", "in place", "other"])
def test_views_that_do_not_flatten(L, gpu, view, place):  # noqa: F811
    rng = np.random.default_rng(3)
    full = torch.from_numpy(rng.standard_normal((6, 7, 6, 64)).astype(np.float32)).bfloat16().to(gpu)
    x = VIEWS[view](full)
    pos = torch.from_numpy(rng.integers(0, 9000, x.shape[:-2]).astype(np.int32)).to(gpu)
    freqs, _ = L.rope_frequencies(32, device=gpu)
    flat = x.contiguous().view(-1, *x.shape[-2:])
    want = L.rope_rotate(flat, pos.view(-1), freqs, first=2).view(x.shape)
    before = full.clone()
    out = None if place == "new" else x if place == "in place" else VIEWS[view](torch.full_like(full, 3.0))
    got = L.rope_rotate(x, pos, freqs, first=2, out=out)
    torch.cuda.synchronize()
    assert L.check_device() == 0
    assert got.shape == x.shape and torch.equal(got, want) and (out is None or got is out)
    if place != "in place":
        assert torch.equal(full, before)
    else:
        VIEWS[view](before).copy_(want)
        assert torch.equal(full, before)


def test_results_in_one_place_are_refused(L, gpu):  # noqa: F811
    x = torch.zeros((3, 4, 2, 64), dtype=torch.bfloat16, device=gpu)
    pos = torch.zeros((3, 4), dtype=torch.int32, device=gpu)
    freqs, _ = L.rope_frequencies(64, device=gpu)
    for out in (x[:1].expand(3, -1, -1, -1), x[:, :1].expand(-1, 4, -1, -1), x[:, :, :1].expand(-1, -1, 2, -1)):
        with pytest.raises((ValueError, L.LkvError)):
            L.rope_rotate(x, pos, freqs, out=out)
        with pytest.raises((ValueError, L.LkvError)):
            L.rope_rotate(out, pos, freqs, out=out)
    assert torch.equal(L.rope_rotate(x[:1].expand(3, -1, -1, -1), pos, freqs), x)
