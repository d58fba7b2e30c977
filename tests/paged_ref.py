"""Paged serving from the definition, in numpy and 64 bits: the reference of the
paged tests. Row by row and token by token; it shares no code with the library."""
from __future__ import annotations

import math

import numpy as np


def round_type(x, dtype):
    """float64 values rounded to a type's grid ("f32", "f16", "bf16")."""
    x = np.asarray(x, np.float64)
    if dtype == "f32":
        return x.astype(np.float32).astype(np.float64)
    if dtype == "f16":
        return x.astype(np.float16).astype(np.float64)
    b = x.astype(np.float32).view(np.uint32).astype(np.uint64)
    b = (b + 0x7fff + ((b >> 16) & 1)) & 0xffff0000
    return b.astype(np.uint32).view(np.float32).astype(np.float64)


HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}

# ------------------------------------------------------------- 4-bit rows


def encode(x):
    """Rows [..., hd] -> codes [..., hd] uint8, scales [..., hd/32] float16, factors [...] float32."""
    x = np.asarray(x, np.float32)
    xb = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    with np.errstate(all="ignore"):
        d = np.abs(xb).max(-1) / np.float32(-8)
        inv = np.where(d != 0, np.float32(1) / np.where(d != 0, d, np.float32(1)), np.float32(0))
        codes = np.clip(np.rint(xb * inv[..., None]), -8, 7) + 8
    top = np.abs(d).max(-1)
    e = np.clip(np.frexp(np.where(top > 0, top, 1))[1] - 1, -126, 127)
    factors = np.where(top > 0, np.ldexp(np.float32(1), e), np.float32(1)).astype(np.float32)
    return (codes.astype(np.uint8).reshape(x.shape), (d / factors[..., None]).astype(np.float16),
            factors)


def decode(codes, scales, factors):
    s = scales.astype(np.float64) * factors.astype(np.float64)[..., None]
    return (codes.astype(np.float64) - 8) * np.repeat(s, 32, -1)


def group_bytes(hd):
    return 2 * (9 * hd + 32)


def code_place(hd, r, e, v):
    """(byte, shift) of element e of row r inside a part."""
    nb, b = hd // 32, e // 32
    if not v:
        j = (r // 8) * nb + b
        return ((j // 4) * 32 + (r % 8) * 4 + e % 32 // 8) * 16 + (j % 4) * 4 + e % 8 // 2, 4 * (e % 2)
    j = (r % 2 + 2 * (r // 8)) * nb + b
    return ((j // 8) * 32 + e % 32 // 4 * 4 + r % 8 // 2) * 16 + (j % 8) * 2 + e % 4 // 2, 4 * (e % 2)


def scale_place(hd, r, b, v):
    nb = hd // 32
    if not v:
        return 8 * hd + 2 * (r * nb + b)
    return 8 * hd + 2 * (((b // 2) * 4 + r % 8 // 2) * 8 + (b % 2) * 4 + r % 2 + 2 * (r // 8))


def put_row(pages, page_rows, hkv, hd, slot, h, x, v):
    """Encode one row of K (v = 0) or V (v = 1) into a uint8 numpy pool."""
    page, at = divmod(slot, page_rows)
    base = ((page * hkv + h) * (page_rows // 16) + at // 16) * group_bytes(hd) + v * (9 * hd + 32)
    r = at % 16
    codes, scales, factor = encode(x)
    for e in range(hd):
        byte, shift = code_place(hd, r, e, v)
        pages[base + byte] = (pages[base + byte] & (0xf0 >> shift)) | (int(codes[e]) << shift)
    for b in range(hd // 32):
        o = base + scale_place(hd, r, b, v)
        pages[o:o + 2] = scales[b:b + 1].view(np.uint8)
    o = base + 9 * hd + 2 * r
    pages[o:o + 2] = (np.array([factor]).view(np.uint32) >> 16).astype(np.uint16).view(np.uint8)


# ------------------------------------------------------------------- plan


def plan(cached, fresh, ring, state, table, page_rows, max_tokens):
    """One step, request by request. Returns a dict of everything fa_page_plan writes."""
    ring, table = list(ring), [list(row) for row in table]
    n, (head, count) = len(ring), state
    taken, wanted, back, lens, cu, slots, pos = 0, 0, [], [], [0], [], []
    for r, (c, f) in enumerate(zip(cached, fresh)):
        used = -(-c // page_rows)
        if f < 0:
            back += table[r][:used]
            lens.append(0)
            cu.append(cu[-1])
            continue
        need = -(-(c + f) // page_rows) - used
        wanted += need
        fits = need == 0 or wanted <= count
        if fits and need:
            for k in range(need):
                table[r][used + k] = ring[(head + wanted - need + k) % n]
            taken = wanted
        lens.append(c + f if fits else c)
        cu.append(cu[-1] + f)
        for p in range(c, c + f):
            pos.append(p)
            slots.append(table[r][p // page_rows] * page_rows + p % page_rows if fits else -1)
    for i, page in enumerate(back):
        ring[(head + count + i) % n] = page
    pad = max_tokens - len(slots)
    return dict(ring=ring, table=table, lens=lens, cu=cu, slots=slots + [-1] * pad,
                positions=pos + [0] * pad,
                state=[(head + taken) % n, count - taken + len(back), wanted - taken])


# ------------------------------------------------------------------- rope


def axes_of(pairs, sections, interleaved):
    n = len(sections)
    if not interleaved:
        return np.repeat(np.arange(n), sections)
    return np.array([i % n if i < n * sections[i % n] else 0 for i in range(pairs)])


def rope(x, positions, inv_freq, axis, adjacent, inverse):
    """x [T][H][hd] float64, positions [A][T] -> rotated, float64."""
    x = np.array(x, np.float64)
    half = len(inv_freq)
    # angles modulo a turn in long integers: far positions lose nothing
    turn = 2 * math.pi
    a = np.array([[math.fmod(int(p) * float(f), turn) for f, p in zip(inv_freq, positions[axis, t])]
                  for t in range(x.shape[0])])[:, None, :]
    if inverse:
        a = -a
    i = np.arange(half)
    lo, hi = (2 * i, 2 * i + 1) if adjacent else (i, i + half)
    u, w = x[..., lo].copy(), x[..., hi].copy()
    x[..., lo] = u * np.cos(a) - w * np.sin(a)
    x[..., hi] = u * np.sin(a) + w * np.cos(a)
    return x


# -------------------------------------------------------------- attention


def attend(q, n_rows, k, v, first, sink, win, scale):
    """Queries q [n][Hq][hd] at positions first.. over rows k, v [L][Hkv][hd] (float64).
    Returns out [n][Hq][hd], lse [Hq][n]."""
    n, hq, hd = q.shape
    g = hq // k.shape[1]
    out, lse = np.zeros(q.shape), np.full((hq, n), -math.inf)
    j = np.arange(n_rows)
    for i in range(n):
        p = first + i
        see = j <= p
        if win > 0:
            see &= (j < sink) | (j > p - win)
        if not see.any():
            continue
        kk, vv = (np.repeat(x[:n_rows][see], g, 1) for x in (k, v))
        s = np.einsum("hd,jhd->hj", q[i], kk) * scale
        m = s.max(-1, keepdims=True)
        w = np.exp(s - m)
        out[i] = np.einsum("hj,jhd->hd", w, vv) / w.sum(-1, keepdims=True)
        lse[:, i] = (m + np.log(w.sum(-1, keepdims=True)))[:, 0]
    return out, lse
