"""Pools of the paged 4-bit cache that are large enough to fill a GPU's CTAs several times over, and their decode in fp64,
both in torch operations on any device.  A row's bytes follow include/lkv.h; nothing of the library is used."""
import math

import numpy as np
import torch

from paged_util import D_ROPE

# The eight codes of a little-endian 32-bit word, in the order of their columns: shift of each nibble.
SHIFTS = (0, 16, 4, 20, 8, 24, 12, 28)


def rope_at(r):
    return r // 2 + -(-(r // 16) // 16) * 16


def _places(lens, page, g, device):
    """(table int32 [B, max_pages] with -1 in unused entries, pages, page and slot of every token, requests laid end to end)."""
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 2
    order = torch.randperm(pages, generator=g, device=device)[:max(1, sum(need))]
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32, device=device)
    where, at = [], 0
    for b, (n, k) in enumerate(zip(lens, need)):
        mine = order[at:at + k]
        table[b, :k] = mine.to(torch.int32)
        at += k
        t = torch.arange(n, device=device)
        where.append(torch.stack([mine[t // page], t % page]) if n else torch.zeros((2, 0), dtype=torch.int64, device=device))
    return table, pages, torch.cat(where, 1)


def make_large(lens, groups, d, page, seed, device, key0=None, exponent=-6):
    """(pool uint8 [pages, page, row bytes], table).  Codes uniform over -7 .. 7, scales n 2^exponent with n in 8 .. 15, RoPE
    keys unit normal; key0(b, t): their first column instead, for the tokens t of request b (values exact in bf16).  Slots
    without a token and unused pages hold 0xFF."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    table, pages, where = _places(lens, page, g, device)
    r, n = groups * d, sum(lens)
    at = rope_at(r)
    rows = torch.zeros((n, at + 2 * D_ROPE), dtype=torch.uint8, device=device)
    nib = torch.randint(1, 16, (2, n, r // 2), generator=g, device=device, dtype=torch.uint8)
    rows[:, :r // 2] = nib[0] | nib[1] << 4
    scales = torch.randint(8, 16, (n, r // 32), generator=g, device=device).double() * 2.0 ** exponent
    rows[:, r // 2:r // 2 + r // 16] = scales.to(torch.bfloat16).view(torch.uint8).view(n, r // 16)
    kpe = torch.randn((n, D_ROPE), generator=g, device=device).to(torch.bfloat16)
    if key0 is not None and n:
        first = torch.cat([key0(b, torch.arange(m, device=device)) for b, m in enumerate(lens)]).double()
        assert torch.equal(first.to(torch.bfloat16).double(), first), "first columns must be exact in bf16"
        kpe[:, 0] = first.to(torch.bfloat16)
    rows[:, at:] = kpe.view(torch.uint8).view(n, 2 * D_ROPE)
    pool = torch.full((pages, page, rows.shape[1]), 0xFF, dtype=torch.uint8, device=device)
    pool[where[0], where[1]] = rows
    return pool, table


def make_queries(B, s_q, H, d, seed, device, std=1.0):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    q = (torch.randn((B, s_q, H, d + D_ROPE), generator=g, device=device) * std).to(torch.bfloat16)
    return q[..., :d].contiguous(), q[..., d:].contiguous()


def decode64(q, q_rope, pool, groups, table, lens, scale):
    """As oracle.paged.paged_decode: out, lse, spread, mass in fp64 (numpy), one request at a time over all its heads."""
    B, S, H, d = q.shape
    dev, r, page = q.device, groups * d, pool.shape[1]
    out, spread = (torch.zeros((B, S, H, d), dtype=torch.float64, device=dev) for _ in range(2))
    lse, mass = torch.full((B, S, H), -math.inf, dtype=torch.float64, device=dev), torch.zeros((B, S, H), dtype=torch.float64, device=dev)
    for b, n in enumerate(lens):
        if n <= 0:
            continue
        rows = pool[table[b, :-(-n // page)].long()].flatten(0, 1)[:n]
        word = rows[:, :r // 2].contiguous().view(torch.int32)
        codes = torch.stack([(word >> k & 15) - 8 for k in SHIFTS], -1).reshape(n, r // 32, 32)
        sc = rows[:, r // 2:r // 2 + r // 16].contiguous().view(torch.bfloat16).double()
        lat = (codes * sc[..., None]).reshape(n, groups, d).transpose(0, 1)                      # [G, n, d]
        kpe = rows[:, rope_at(r):rope_at(r) + 2 * D_ROPE].contiguous().view(torch.bfloat16).double()
        qn = q[b].double().view(S, groups, H // groups, d).transpose(0, 1).reshape(groups, -1, d)   # [G, S * heads, d]
        qr = q_rope[b].double().view(S, groups, H // groups, D_ROPE).transpose(0, 1).reshape(groups, -1, D_ROPE)
        s = scale * (qn @ lat.transpose(1, 2) + qr @ kpe.T)
        size = scale * (qn.abs() @ lat.abs().transpose(1, 2) + qr.abs() @ kpe.abs().T)
        new = torch.arange(S, device=dev).repeat_interleave(H // groups)                         # the new token of a row
        hidden = torch.arange(n, device=dev) > (n - S + new)[:, None]
        s, size = s.masked_fill(hidden, -math.inf), size.masked_fill(hidden, 0.0)
        top = s.amax(-1)
        l = torch.where(top == -math.inf, top, torch.logsumexp(s, -1))
        p = torch.where(hidden, 0.0, torch.exp(s - torch.where(l == -math.inf, 0.0, l)[..., None]))
        back = lambda x: x.reshape(groups, S, H // groups, *x.shape[2:]).transpose(0, 1).reshape(S, H, *x.shape[2:])  # noqa: E731
        lse[b], mass[b] = back(l), back(size.amax(-1))
        out[b], spread[b] = back(p @ lat), back(p @ lat.abs())
    return tuple(x.cpu().numpy() for x in (out, lse, spread, mass))


def tiles(lens):
    return sum(-(-n // 128) for n in lens if n > 0)


def ragged(live, mean, seed, longest, idle=3):
    """`live` lengths around `mean` (1 among them), a few idle slots, and one long request."""
    rng = np.random.default_rng(seed)
    lens = [max(1, int(v)) for v in rng.exponential(mean, live - 2)] + [1, longest] + [0] * idle
    return [lens[i] for i in rng.permutation(len(lens))]
