"""Cases for measuring the operators of a paged 4-bit latent cache: rotary positions (rope_rotate), the
append that rotates, quantises and scatters new rows (paged_append_int4), and decode attention over
the cache (paged_decode_int4).

With `own` false run() computes each operator in plain torch operations in fp32 (angles in fp64);
with `own` true it makes the library's calls.  exact() is the definition in fp64.

A cache row of r latent columns and d_rope RoPE columns (one token):
  bytes [0, r/2)   4-bit codes, u = code + 8, code in [-7, 7].  Eight columns share a 32-bit little-endian
                   word: column 2i of the eight in bits 4i..4i+3, column 2i+1 in bits 16+4i..19+4i
  then r/32        bf16 scales, one for each 32 columns (the field padded to a multiple of 16 bytes)
  then d_rope      bf16 values, the rotated RoPE key
"""
import math
import random

import torch

own = False

BLOCK = 32          # latent columns that share a scale
D_ROPE = 64         # RoPE width of the decode workloads


# ------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one user, a few tokens into an answer: a call that is all latency
        {"name": "decode_one", "op": "decode", "d": 128, "groups": 8, "heads": 128, "s_q": 1, "batch": 1, "len_lo": 37,
         "len_hi": 37, "page": 16},
        # a small model's chat batch: 8 heads for each tied group, ragged lengths, some slots idle
        {"name": "decode_chat", "op": "decode", "d": 128, "groups": 4, "heads": 32, "s_q": 1, "batch": 24, "len_lo": 0,
         "len_hi": 2500, "page": 32},
        # the GTA workload: 64 requests of 8192 tokens, two new tokens each
        {"name": "decode_gta", "op": "decode", "d": 128, "groups": 8, "heads": 128, "s_q": 2, "batch": 64, "len_lo": 8192,
         "len_hi": 8192, "page": 64},
        # wide groups (2 x 64 heads), lengths from tens to tens of thousands, pages that end inside a tile
        {"name": "decode_varlen", "op": "decode", "d": 128, "groups": 2, "heads": 128, "s_q": 1, "batch": 32, "len_lo": 64,
         "len_hi": 20000, "page": 48},
        # the long-context GLA workload: 8 requests of 131072 tokens, two latent groups of 256
        {"name": "decode_gla_long", "op": "decode", "d": 256, "groups": 2, "heads": 128, "s_q": 1, "batch": 8,
         "len_lo": 131072, "len_hi": 131072, "page": 64},
        # the MLA workload: one latent of 512 for all 128 heads
        {"name": "decode_mla", "op": "decode", "d": 512, "groups": 1, "heads": 128, "s_q": 1, "batch": 64, "len_lo": 4096,
         "len_hi": 4096, "page": 64},
        # the new rows of one decode step of the GTA workload
        {"name": "append_step", "op": "append", "r": 1024, "batch": 64, "new_lo": 2, "new_hi": 2, "ctx": 200, "page": 64,
         "interleaved": False, "factor": 1.0},
        # prompts of different lengths entering an MLA cache, positions scaled to a longer context
        {"name": "append_prompts", "op": "append", "r": 512, "batch": 24, "new_lo": 500, "new_hi": 6000, "ctx": 100,
         "page": 48, "interleaved": True, "factor": 16.0},
        # the queries of one decode step of the GTA workload, far into the context
        {"name": "rope_step", "op": "rope", "tokens": 128, "heads": 128, "dim": 64, "first": 0, "rot": 64,
         "interleaved": False, "inverse": False, "dtype": "bf16", "max_pos": 131072, "factor": 1.0},
        # a prompt's queries: the last 64 of 192 columns of each head, interleaved pairs
        {"name": "rope_prompt", "op": "rope", "tokens": 8192, "heads": 128, "dim": 192, "first": 128, "rot": 64,
         "interleaved": True, "inverse": False, "dtype": "bf16", "max_pos": 8192, "factor": 1.0},
        # the gradient of a rotation in fp32, odd sizes, positions scaled to a longer context
        {"name": "rope_grad_fp32", "op": "rope", "tokens": 3001, "heads": 12, "dim": 96, "first": 0, "rot": 48,
         "interleaved": False, "inverse": True, "dtype": "fp32", "max_pos": 1000000, "factor": 8.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "append", "rope"])
    if op == "decode":
        d = rng.choice([128, 128, 256, 512])
        groups = rng.choice([g for g in (1, 2, 4, 8) if g * d <= 1024])
        per = rng.choice([1, 2, 3, 4, 5, 8, 12, 16, 32, 64]) if d < 512 else rng.choice([8, 16, 64, 128])
        per = min(per, 128 // groups)
        hi = _log(rng, 40, 131072)
        # about 2^19 tokens x 1024 columns x heads at most, as in the largest listed case
        most = max(1, min(64, int(2 ** 19 / hi), int(2 ** 29 / (hi * groups * d))))
        lo = rng.choice([0, 1, max(1, hi // 8), hi])
        return {"op": "decode", "d": d, "groups": groups, "heads": groups * per, "s_q": rng.choice([1, 2]),
                "batch": rng.randint(1, most), "len_lo": lo, "len_hi": hi,
                "page": rng.choice([1, 16, 32, 48, 64, 100, 128, 256])}
    if op == "append":
        hi = _log(rng, 1, 4000)
        return {"op": "append", "r": BLOCK * rng.choice([1, 4, 8, 16, 20, 32]), "batch": rng.randint(1, max(1, min(64, 100000 // hi))),
                "new_lo": rng.choice([0, 1, hi]), "new_hi": hi, "ctx": rng.randint(0, 300),
                "page": rng.choice([1, 16, 48, 64, 100]), "interleaved": rng.random() < 0.5,
                "factor": rng.choice([1.0, 4.0, 16.0])}
    dim = rng.choice([64, 80, 96, 128, 192])
    rot = rng.choice([v for v in (32, 48, 64, 96, 128) if v <= dim])
    heads = rng.choice([1, 5, 12, 32, 128])
    return {"op": "rope", "tokens": _log(rng, 1, max(2, 200_000_000 // (heads * dim))), "heads": heads, "dim": dim,
            "first": rng.choice([0, dim - rot]), "rot": rot, "interleaved": rng.random() < 0.5,
            "inverse": rng.random() < 0.5, "dtype": rng.choice(["bf16", "fp32"]), "max_pos": _log(rng, 100, 1000000),
            "factor": rng.choice([1.0, 8.0])}


def _spread(case, lo, hi):
    """Whole numbers between lo and hi, one for each request, evenly over their logarithm, in a mixed order."""
    n = case["batch"]
    if lo == hi:
        return [hi] * n
    a = max(lo, 1)
    at = [int(round(a * (hi / a) ** (i / max(1, n - 1)))) for i in range(n)]
    at[-1] = hi
    if lo == 0 and n > 2:
        at[0] = at[1] = 0
    random.Random(n * 7919 + hi).shuffle(at)
    return at


def _lengths(case):
    return _spread(case, case["len_lo"], case["len_hi"])


def _row_bytes(r, d_rope):
    return r // 2 + (r // 16 + 15) // 16 * 16 + 2 * d_rope


def _scale_at(r):
    return r // 2


def _rope_at(r, d_rope):
    return _row_bytes(r, d_rope) - 2 * d_rope


# --------------------------------------------------------------------------------- what a program has

def _frequencies(rot, factor, device):
    """base^(-2i/rot) radians a position; for factor > 1 the slow ones are divided by it (a ramp between 1 and 32
    turns over a context of 4096) and the pairs are scaled by the gain."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    if factor == 1.0:
        return f, 1.0
    keep = ((4096.0 * f / (2 * math.pi) - 1.0) / 31.0).clamp(0.0, 1.0)
    return f * (keep + (1.0 - keep) / factor), 1.0 + 0.1 * math.log(factor)


def _pages(lens, page, g, device):
    """A block table over shuffled pages; entries that no token needs hold -1."""
    need = [-(-n // page) for n in lens]
    total = max(1, sum(need))
    order = torch.randperm(total + 3, generator=g, device=device).to(torch.int32)[:total]
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32, device=device)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, total + 3


def _normal(shape, std, g, device, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device=device) * std).to(dtype)


def _quantise(x):
    """[n, r] -> codes [n, r] (whole fp32 values), scales [n, r / 32] fp32."""
    n, r = x.shape
    v = x.float().reshape(n, r // BLOCK, BLOCK)
    amax = v.abs().amax(-1)
    frac, exp = torch.frexp(amax)
    m = (frac * 256).to(torch.int32)                   # the 8 significant bits of a bf16 value: amax = m 2^(exp - 8)
    low, high = (m + 13) // 14, (m + 27) // 28         # the least n with 7 n 2 >= m, with 7 n 4 >= m
    two = (exp + 120 << 23).view(torch.float32)        # 2^(exp - 7), by its bits: pow() need not be exact
    s = torch.where(low <= 15, low * two, high * (2 * two))
    s = torch.where(amax > 0, s, torch.zeros_like(s))
    code = torch.round(v / torch.where(s > 0, s, torch.ones_like(s))[..., None]).clamp(-7, 7)
    return code.reshape(n, r), s


def _pack(code):
    """Whole values [n, r] in [-7, 7] -> uint8 [n, r / 2]."""
    n, r = code.shape
    u = (code + 8).to(torch.int32).reshape(n, r // 8, 8)
    return torch.stack([u[..., 0] | u[..., 2] << 4, u[..., 4] | u[..., 6] << 4,
                        u[..., 1] | u[..., 3] << 4, u[..., 5] | u[..., 7] << 4], -1).to(torch.uint8).reshape(n, r // 2)


def _rows_of(x, kpe):
    """Cache rows of latent x [n, r] and (rotated) keys kpe [n, d_rope], as bytes."""
    n, r = x.shape
    code, s = _quantise(x)
    rows = torch.zeros((n, _row_bytes(r, kpe.shape[1])), dtype=torch.uint8, device=x.device)
    rows[:, :r // 2] = _pack(code)
    rows[:, _scale_at(r):_scale_at(r) + r // 16] = s.to(torch.bfloat16).view(torch.uint8).reshape(n, -1)
    rows[:, _rope_at(r, kpe.shape[1]):] = kpe.to(torch.bfloat16).contiguous().view(torch.uint8).reshape(n, -1)
    return rows


def prepare(case, seed):
    device = torch.device("cuda")
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    if case["op"] == "rope":
        dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        x = _normal((case["tokens"], case["heads"], case["dim"]), 1.0, g, device, dtype)
        pos = torch.randint(0, case["max_pos"], (case["tokens"],), generator=g, device=device, dtype=torch.int32)
        freqs, gain = _frequencies(case["rot"], case["factor"], device)
        return {"case": case, "x": x, "pos": pos, "freqs": freqs, "gain": gain}
    if case["op"] == "append":
        r = case["r"]
        new = _spread(case, case["new_lo"], case["new_hi"])
        lens = [n + (case["ctx"] * (b % 5)) // 4 for b, n in enumerate(new)]
        table, pages = _pages(lens, case["page"], g, device)
        cu = torch.tensor([0] + new, device=device).cumsum(0).to(torch.int32)
        rows = _normal((sum(new), r + D_ROPE), 1.0 / math.sqrt(192.0), g, device)
        pool = torch.zeros((pages, case["page"], _row_bytes(r, D_ROPE)), dtype=torch.uint8, device=device)
        freqs, gain = _frequencies(D_ROPE, case["factor"], device)
        return {"case": case, "rows": rows, "pool": pool, "table": table, "cu": cu, "freqs": freqs, "gain": gain,
                "lens": torch.tensor(lens, dtype=torch.int32, device=device), "held": torch.empty_like(rows)}
    d, G, H, s_q, B = case["d"], case["groups"], case["heads"], case["s_q"], case["batch"]
    lens = _lengths(case)
    table, pages = _pages(lens, case["page"], g, device)
    n, width = pages * case["page"], _row_bytes(G * d, D_ROPE)
    pool = torch.empty((n, width), dtype=torch.uint8, device=device)
    step = 65536
    for at in range(0, n, step):                       # states of unit variance, as a norm leaves them
        k = min(step, n - at)
        pool[at:at + k] = _rows_of(_normal((k, G * d), 1.0, g, device), _normal((k, D_ROPE), 1.0, g, device))
    pool = pool.reshape(pages, case["page"], width)
    for b, m in enumerate(lens):                       # slots behind a sequence's end were never written
        if m % case["page"]:
            pool[table[b, m // case["page"]].long(), m % case["page"]:] = 0xFF
    q = _normal((B, s_q, H, d), 1.0, g, device)
    q_rope = _normal((B, s_q, H, D_ROPE), 1.0, g, device)
    return {"case": case, "q": q, "q_rope": q_rope, "pool": pool, "table": table,
            "lens": torch.tensor(lens, dtype=torch.int32, device=device)}


# ------------------------------------------------------------------------------------------ one pass

def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import latent_kv_cache_split_b200 as lkv
        if op == "rope":
            return lkv.rope_rotate(s["x"], s["pos"], s["freqs"], first=case["first"], interleaved=case["interleaved"],
                                   inverse=case["inverse"], gain=s["gain"])
        if op == "append":
            lkv.paged_append_int4(s["rows"], s["pool"], case["r"], s["table"], s["lens"], cu_new=s["cu"], freqs=s["freqs"],
                                  gain=s["gain"], interleaved=case["interleaved"], rows_out=s["held"])
            return _appended(s, s["held"])
        out, lse = lkv.paged_decode_int4(s["q"], s["q_rope"], s["pool"], case["groups"], s["table"], s["lens"],
                                         1.0 / math.sqrt(case["d"] + D_ROPE))
        return {"out": out, "lse": lse}
    if op == "rope":
        return _plain_rope(s["x"], s["pos"], s["freqs"], s["gain"], case["first"], case["interleaved"], case["inverse"])
    if op == "append":
        return _plain_append(s)
    return _plain_decode(s)


def _appended(s, held):
    """The new rows as the cache holds them (values), and the cache itself in views of its fields."""
    r, pool = s["case"]["r"], s["pool"]
    at, end = _scale_at(r), _scale_at(r) + r // 16
    return {"held": held, "codes": pool[..., :at], "scales": pool[..., at:end].view(torch.bfloat16),
            "kpe": pool[..., _rope_at(r, D_ROPE):].view(torch.bfloat16)}


def _plain_rope(x, pos, freqs, gain, first, interleaved, inverse):
    rot = 2 * freqs.numel()
    angle = pos.double()[:, None] * freqs
    cos, sin = (gain * angle.cos()).float()[:, None], (gain * angle.sin()).float()[:, None]
    sin = -sin if inverse else sin
    v = x[..., first:first + rot].float()
    a, b = (v[..., 0::2], v[..., 1::2]) if interleaved else (v[..., :rot // 2], v[..., rot // 2:])
    a, b = a * cos - b * sin, a * sin + b * cos
    v = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    out = x.clone()
    out[..., first:first + rot] = v.to(x.dtype)
    return out


def _plain_append(s):
    case, r, page = s["case"], s["case"]["r"], s["case"]["page"]
    rows, cu, n = s["rows"], s["cu"].long(), s["rows"].shape[0]
    t = torch.arange(n, device=rows.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    pos = s["lens"].long()[b] - (cu[b + 1] - t)
    kpe = _plain_rope(rows[:, None, r:], pos, s["freqs"], s["gain"], 0, case["interleaved"], False)[:, 0]
    packed = _rows_of(rows[:, :r], kpe)
    s["pool"][s["table"][b, pos // page].long(), pos % page] = packed
    code, scale = _quantise(rows[:, :r])
    value = code * scale.repeat_interleave(BLOCK, 1)
    return _appended(s, torch.cat([value.to(torch.bfloat16), kpe], 1))


def _unpack(c):
    """uint8 [..., r / 2] -> fp32 [..., r]: the codes' whole values."""
    c = c.reshape(*c.shape[:-1], c.shape[-1] // 4, 4)
    lo, hi = c & 15, c >> 4
    u = torch.stack([lo[..., 0], lo[..., 2], hi[..., 0], hi[..., 2], lo[..., 1], lo[..., 3], hi[..., 1], hi[..., 3]], -1)
    return u.float().flatten(-2) - 8


def _plain_decode(s):
    case = s["case"]
    d, G, H, s_q, B, page = case["d"], case["groups"], case["heads"], case["s_q"], case["batch"], case["page"]
    r, lens = G * d, s["lens"].long()
    T = s["table"].shape[1] * page
    at = s["table"].clamp(min=0).long()
    t = torch.arange(T, device=lens.device)
    there = (t < lens[:, None])[..., None]
    rows = s["pool"][at].reshape(B, T, -1)
    scale = torch.where(there, rows[..., _scale_at(r):_scale_at(r) + r // 16].view(torch.bfloat16).float(), 0.0)
    c = _unpack(rows[..., :r // 2]).reshape(B, T, r // BLOCK, BLOCK) * scale[..., None]
    c = c.reshape(B, T, G, d).transpose(1, 2)                                           # [B, G, T, d]
    kpe = torch.where(there, rows[..., _rope_at(r, D_ROPE):].view(torch.bfloat16).float(), 0.0)
    q = s["q"].float().reshape(B, s_q, G, H // G, d).transpose(1, 2).reshape(B, G, -1, d)
    q_rope = s["q_rope"].float().reshape(B, s_q, G, H // G, D_ROPE).transpose(1, 2).reshape(B, G, -1, D_ROPE)
    score = (q @ c.transpose(2, 3) + q_rope @ kpe.transpose(1, 2)[:, None]) / math.sqrt(d + D_ROPE)
    last = lens[:, None] - s_q + torch.arange(s_q, device=lens.device)                  # newest key of each query
    seen = (t <= last[..., None])[:, None, :, None, :]
    score = score.reshape(B, G, s_q, H // G, T).masked_fill(~seen, -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    out = (p.reshape(B, G, -1, T) @ c).reshape(B, G, s_q, H // G, d) / total.clamp(min=1e-30)
    lse = (top + torch.log(total))[..., 0]
    return {"out": out.transpose(1, 2).reshape(B, s_q, H, d).to(torch.bfloat16),
            "lse": lse.transpose(1, 2).reshape(B, s_q, H)}


# ------------------------------------------------------------------------------------------ the work

def work(case):
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"]
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * n * case["dim"] * size + 4 * case["tokens"] + 4 * case["rot"], "flops": 3 * n * case["rot"]}
    if case["op"] == "append":
        n, r = sum(_spread(case, case["new_lo"], case["new_hi"])), case["r"]
        # rows in, rows of the cache out, the held values out
        return {"bytes": n * (4 * (r + D_ROPE) + _row_bytes(r, D_ROPE)), "flops": n * (4 * r + 3 * D_ROPE)}
    tokens, r = sum(_lengths(case)), case["groups"] * case["d"]
    q = case["batch"] * case["s_q"] * case["heads"]
    used = r // 2 + r // 16 + 2 * D_ROPE
    return {"bytes": tokens * used + q * (4 * case["d"] + 2 * D_ROPE + 4),
            "flops": 2 * tokens * case["s_q"] * case["heads"] * (2 * case["d"] + D_ROPE)}


# --------------------------------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s["x"], s["pos"], case, s["freqs"], s["gain"], case["first"], case["inverse"])
    if case["op"] == "append":
        return _exact_append(s)
    return _exact_decode(s)


def _exact_rope(x, pos, case, freqs, gain, first, inverse):
    """Each pair as a complex number, multiplied by gain * exp(+-i * angle)."""
    rot = 2 * freqs.numel()
    y = x.double()
    v = y[..., first:first + rot]
    half = rot // 2
    pair = v.unflatten(-1, (half, 2)) if case["interleaved"] else v.unflatten(-1, (2, half)).transpose(-1, -2)
    turn = torch.polar(torch.full_like(freqs, gain).expand(pos.numel(), half),
                       (-1.0 if inverse else 1.0) * torch.outer(pos.double(), freqs))
    pair = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn[:, None, :])
    y[..., first:first + rot] = (pair if case["interleaved"] else pair.transpose(-1, -2)).flatten(-2)
    return y


def _exact_append(s):
    case, page, r = s["case"], s["case"]["page"], s["case"]["r"]
    rows, table, lens, cu = s["rows"], s["table"].tolist(), s["lens"].tolist(), s["cu"].tolist()
    n = rows.shape[0]
    where = [(b, lens[b] - (cu[b + 1] - cu[b]) + j) for b in range(len(lens)) for j in range(cu[b + 1] - cu[b])]
    pos = torch.tensor([p for _, p in where], device=rows.device)
    kpe = _exact_rope(rows[:, None, r:], pos, case, s["freqs"], s["gain"], 0, False)[:, 0]
    v = rows[:, :r].double().reshape(n, -1, BLOCK)
    amax = v.abs().amax(-1)
    # the 4-significant-bit numbers around amax / 7, and the smallest of them that reaches it
    e = torch.floor(torch.log2(amax.clamp(min=1e-300) / 7)).long() - 3
    grid = torch.arange(7, 18, device=rows.device, dtype=torch.float64) * (e + 1023 << 52).view(torch.float64)[..., None]
    grid = torch.where((torch.arange(7, 18, device=rows.device) == 17), torch.full_like(grid, math.inf), grid)
    scale = torch.where(7 * grid >= amax[..., None], grid, torch.full_like(grid, math.inf)).amin(-1)
    scale = torch.where(amax > 0, scale, torch.zeros_like(scale))
    code = torch.where(scale[..., None] > 0, torch.round(v / scale.clamp(min=1e-300)[..., None]), torch.zeros_like(v))
    held = torch.cat([(code * scale[..., None]).reshape(n, r), kpe], 1)
    pages, rope = s["pool"].shape[0], rows.shape[1] - r
    scales = torch.zeros((pages, page, r // BLOCK), dtype=torch.float64, device=rows.device)
    keys = torch.zeros((pages, page, rope), dtype=torch.float64, device=rows.device)
    if n:
        at = torch.tensor([table[b][p // page] * page + p % page for b, p in where], device=rows.device)
        scales.view(-1, r // BLOCK)[at] = scale
        keys.view(-1, rope)[at] = kpe
    return {"held": held, "codes": None, "scales": scales, "kpe": keys}


def _exact_decode(s):
    case = s["case"]
    d, G, H, s_q, B, page = case["d"], case["groups"], case["heads"], case["s_q"], case["batch"], case["page"]
    r, dev = G * d, s["q"].device
    out = torch.zeros((B, s_q, H, d), dtype=torch.float64, device=dev)
    lse = torch.full((B, s_q, H), -math.inf, dtype=torch.float64, device=dev)
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        used = s["table"][b, :-(-n // page)].long()
        rows = s["pool"][used].flatten(0, 1)[:n]
        word = rows[:, :r // 2].contiguous().view(torch.int32)                          # eight codes each
        nib = torch.stack([word >> k & 15 for k in (0, 16, 4, 20, 8, 24, 12, 28)], -1)
        scale = rows[:, r // 2:r // 2 + r // 16].contiguous().view(torch.bfloat16).double()
        c = ((nib.reshape(n, r // BLOCK, BLOCK) - 8) * scale[..., None]).reshape(n, G, d)
        kpe = rows[:, _rope_at(r, D_ROPE):].contiguous().view(torch.bfloat16).double()
        for i in range(s_q):
            m = n - s_q + i + 1
            if m <= 0:
                continue
            q, q_rope = s["q"][b, i].double().view(G, H // G, d), s["q_rope"][b, i].double()
            score = torch.einsum("ghd,tgd->ght", q, c[:m]).reshape(H, m) + q_rope @ kpe[:m].T
            score = score / math.sqrt(d + D_ROPE)
            lse[b, i] = torch.logsumexp(score, -1)
            p = torch.exp(score - lse[b, i, :, None]).view(G, H // G, m)
            out[b, i] = torch.einsum("ght,tgd->ghd", p, c[:m]).reshape(H, d)
    return {"out": out, "lse": lse}
