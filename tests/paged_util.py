"""Seeded inputs for the paged 4-bit cache, packed by the oracle, and the tolerances of its decode.

Rounding: a bf16 rounding is off by at most 2^-8 of the value, an fp32 one by 2^-24.
* A score is a sum of d + d_rope exact products in fp32 (any order): off by at most (d + d_rope) 2^-23 of the sum of
  their magnitudes (2^-23, not 2^-24, since a tensor core may drop the bits below its accumulator instead of rounding),
  `mass` being the largest such sum over the keys.  The exponent's argument and 2^x add 2^-20 relative.  So
  weights are off by delta = (d + d_rope) 2^-23 mass + 2^-20 (1 + the largest |argument|), argument <= 2 mass.
* lse moves by at most delta, and is stored in fp32.
* out = sum p v / sum p: the weights' rounding to bf16 moves it by at most 2^-8 sum p |v| (spread), delta by 2 delta
  spread, the fp32 sum over n keys by n 2^-23 spread, and the result's rounding by 2^-8 |out|."""
import numpy as np
import torch

from oracle import paged

D_ROPE = 64


def bits(t):
    return t.contiguous().view(torch.int16).numpy().view(np.uint16)


def make_pool(rng, lens, groups, d, page, extra_pages=2, junk=0xFF, std=1.0, max_pages=None):
    """(pool uint8 [pages, page, row bytes], table int32 [B, max_pages]): rows quantised and packed by the oracle, pages
    shuffled, every slot that holds no token and every unused page filled with `junk`, unused table entries -1."""
    r = groups * d
    need = [-(-int(n) // page) for n in lens]
    pages = sum(need) + extra_pages
    order = rng.permutation(pages)
    table = np.full((len(lens), max_pages or max(1, max(need))), -1, dtype=np.int32)
    pool = np.full((pages, page, paged.row_bytes(r, D_ROPE)), junk, dtype=np.uint8)
    at = 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        if n:
            x = torch.from_numpy((rng.standard_normal((int(n), r + D_ROPE)) * std).astype(np.float32)).bfloat16()
            # codes and scales drawn as such: the quantiser has its own tests
            codes = rng.integers(-7, 8, (int(n), r))
            scales = rng.integers(8, 16, (int(n), r // 32)) * 2.0 ** (rng.integers(-7, -4, (int(n), r // 32))) * std
            rows = paged.pack_rows(codes, scales, bits(x[:, r:]), D_ROPE)
            for t in range(int(n)):
                pool[table[b, t // page], t % page] = rows[t]
    return pool, table


def queries(rng, B, s_q, H, d, std=1.0):
    q = torch.from_numpy((rng.standard_normal((B, s_q, H, d + D_ROPE)) * std).astype(np.float32)).bfloat16()
    return q[..., :d].contiguous(), q[..., d:].contiguous()


def check_decode(out, lse, ref, d, n_max, label=""):
    """Apply the tolerances of this module's docstring; ref is paged.paged_decode's result."""
    o, l = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    r_out, r_lse, spread, mass = ref
    empty = np.isneginf(r_lse)
    assert np.array_equal(np.isneginf(l), empty), f"{label}: wrong rows are empty"
    assert (o[empty] == 0).all(), f"{label}: an empty row is not 0"
    assert np.isfinite(o).all() and np.isfinite(l[~empty]).all(), f"{label}: non-finite"
    delta = (d + D_ROPE) * 2.0 ** -23 * mass + 2.0 ** -20 * (1 + 2 * mass)
    tol = (2.0 ** -8 + 2 * delta[..., None] + n_max * 2.0 ** -23) * spread + 2.0 ** -8 * np.abs(r_out) + 1e-30
    over = np.abs(o - r_out) / tol
    assert over.max() <= 1, f"{label}: out is {over.max():.2f} of the tolerance at {np.unravel_index(over.argmax(), over.shape)}"
    l, r_lse, delta = l[~empty], r_lse[~empty], delta[~empty]
    el = np.abs(l - r_lse) / (delta + 2.0 ** -22 * (1 + np.abs(r_lse)))
    assert not el.size or el.max() <= 1, f"{label}: lse is {el.max():.2f} of the tolerance"
    return float(over.max()), float(el.max()) if el.size else 0.0
