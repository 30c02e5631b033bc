"""Rotary positions, 4-bit cache rows and decode over a paged pool, in fp64 (and, for the codes, in
exact rational arithmetic).

TEST INFRASTRUCTURE ONLY, like the rest of oracle/: the library never imports it.

The pages describe none of these; the definitions are the library's own (include/lkv.h):
* a pair (a, b) at position p with frequency f and gain g becomes g (a cos pf - b sin pf),
  g (a sin pf + b cos pf); the inverse negates the angle;
* 32 latent columns share a scale, the smallest n 2^k (n in 8 .. 15) that is at least amax / 7 (0 where
  amax < 2^-100); a code is x / scale rounded to the nearest integer, ties to even;
* token t of request b is row t % page_size of page table[b, t // page_size]; the rest is the decode of
  attend.py with a group's state as key and value.
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np

from .attend import _f64

__all__ = ["rope_rotate", "block_scale", "quantize_rows", "pack_codes", "unpack_codes", "row_bytes", "pack_rows",
           "paged_decode"]

BLOCK = 32


def rope_rotate(x, positions, freqs, first=0, interleaved=False, inverse=False, gain=1.0):
    """x [n, heads, d] -> float64 of the same shape."""
    y = _f64(x).copy()
    f = np.asarray(freqs, dtype=np.float64)
    half = f.size
    for t, p in enumerate(np.asarray(positions).reshape(-1)):
        ang = float(p) * f
        c, s = gain * np.cos(ang), gain * np.sin(ang) * (-1.0 if inverse else 1.0)
        for i in range(half):
            i0, i1 = (first + 2 * i, first + 2 * i + 1) if interleaved else (first + i, first + i + half)
            a, b = y[t, :, i0].copy(), y[t, :, i1].copy()
            y[t, :, i0] = a * c[i] - b * s[i]
            y[t, :, i1] = a * s[i] + b * c[i]
    return y


def block_scale(amax: float) -> Fraction:
    """The scale of a block whose largest magnitude is amax, by trying every n 2^k upwards."""
    a = Fraction(amax)
    if a < Fraction(1, 2 ** 100):
        return Fraction(0)
    k = -130
    while 7 * 15 * Fraction(2) ** k < a:
        k += 1
    for n in range(8, 16):
        if 7 * n * Fraction(2) ** k >= a:
            return n * Fraction(2) ** k
    raise AssertionError


def _round_half_even(q: Fraction) -> int:
    return round(q)          # Python rounds a Fraction to the nearest integer, ties to even


def quantize_rows(x):
    """Latent rows [n, r] (stored bf16 values) -> codes int64 [n, r], scales float64 [n, r / 32]."""
    v = _f64(x)
    n, r = v.shape
    codes = np.zeros((n, r), dtype=np.int64)
    scales = np.zeros((n, r // BLOCK))
    for t in range(n):
        for j in range(r // BLOCK):
            blk = v[t, j * BLOCK:(j + 1) * BLOCK]
            s = block_scale(float(np.abs(blk).max()))
            scales[t, j] = float(s)
            if s:
                codes[t, j * BLOCK:(j + 1) * BLOCK] = [_round_half_even(Fraction(float(e)) / s) for e in blk]
    return codes, scales


def pack_codes(codes):
    """[n, r] in [-7, 7] -> uint8 [n, r / 2], by the bit positions of the format."""
    n, r = codes.shape
    out = np.zeros((n, r // 8), dtype=np.uint32)
    for e in range(8):
        out |= ((codes[:, e::8] + 8).astype(np.uint32) << np.uint32(4 * (e // 2) + 16 * (e % 2)))
    return out.view(np.uint8).reshape(n, r // 2)


def unpack_codes(packed):
    """uint8 [..., r / 2] -> int64 codes [..., r]."""
    w = np.ascontiguousarray(packed).view(np.uint32)
    out = np.zeros(w.shape[:-1] + (w.shape[-1] * 8,), dtype=np.int64)
    for e in range(8):
        out[..., e::8] = ((w >> np.uint32(4 * (e // 2) + 16 * (e % 2))) & np.uint32(15)).astype(np.int64) - 8
    return out


def row_bytes(r, d_rope):
    return r // 2 + -(-(r // 16) // 16) * 16 + 2 * d_rope


def _bf16_bits(v):
    b = np.ascontiguousarray(v, dtype=np.float32).view(np.uint32)
    assert not np.any(b & 0xFFFF), "not a bf16 value"
    return (b >> 16).astype(np.uint16)


def pack_rows(codes, scales, kpe_bits, d_rope):
    """uint8 rows of codes [n, r], scales [n, r / 32] and the RoPE key's bf16 bit patterns [n, d_rope]."""
    n, r = codes.shape
    rows = np.zeros((n, row_bytes(r, d_rope)), dtype=np.uint8)
    rows[:, :r // 2] = pack_codes(codes)
    rows[:, r // 2:r // 2 + r // 16] = _bf16_bits(scales).view(np.uint8).reshape(n, -1)
    if d_rope:
        rows[:, -2 * d_rope:] = np.ascontiguousarray(kpe_bits, dtype=np.uint16).view(np.uint8).reshape(n, -1)
    return rows


def _bf16_values(bits):
    return (np.ascontiguousarray(bits).astype(np.uint32) << np.uint32(16)).view(np.float32).astype(np.float64)


def paged_decode(q, q_rope, pool, groups, table, seq_lens, scale):
    """q [B, s_q, h_q, d], q_rope [B, s_q, h_q, d_rope], pool uint8 [pages, page_size, >= row bytes].

    Returns out, lse (float64; 0 and -inf for a query that sees nothing) and, to derive tolerances from,
    spread = sum_t p_t |v_t| for every output and mass = max_t scale sum_c |q_c k_c| for every query."""
    pool = np.asarray(pool)
    B, S, H, d = q.shape
    dr = q_rope.shape[-1]
    r, hpg = groups * d, H // groups
    out, spread = np.zeros((B, S, H, d)), np.zeros((B, S, H, d))
    lse, mass = np.full((B, S, H), -np.inf), np.zeros((B, S, H))
    page = pool.shape[1]
    for b in range(B):
        n = int(seq_lens[b])
        rows = [pool[int(table[b][t // page]), t % page] for t in range(n)]
        if not rows:
            continue
        rows = np.stack(rows)
        sc = _bf16_values(rows[:, r // 2:r // 2 + r // 16].copy().view(np.uint16))
        lat = (unpack_codes(rows[:, :r // 2]).reshape(n, r // BLOCK, BLOCK) * sc[..., None]).reshape(n, groups, d)
        at = row_bytes(r, dr) - 2 * dr
        kpe = _bf16_values(rows[:, at:at + 2 * dr].copy().view(np.uint16))
        for i in range(S):
            m = n - S + i + 1
            if m <= 0:
                continue
            for h in range(H):
                c = lat[:m, h // hpg]
                qn, qr = _f64(q[b, i, h]), _f64(q_rope[b, i, h])
                s = scale * (c @ qn + kpe[:m] @ qr)
                top = s.max()
                e = np.exp(s - top)
                lse[b, i, h] = top + np.log(e.sum())
                p = e / e.sum()
                out[b, i, h], spread[b, i, h] = p @ c, p @ np.abs(c)
                mass[b, i, h] = scale * (np.abs(c) @ np.abs(qn) + np.abs(kpe[:m]) @ np.abs(qr)).max()
    return out, lse, spread, mass
