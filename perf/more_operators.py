"""Attention with changed scores, for training and for serving, and the paged append that rotates on the way:
their plain forms in elementary torch operations, the calls of the library that compute the same, and their results
from the definition in 64 bits.

kind "packed"  attention of documents packed one behind another
kind "grad"    its gradient: dq, dk, dv from dout
kind "paged"   attention of ragged queries over 4-bit pages
kind "append"  q and k rotated to their positions, K and V into 4-bit pages, then the requests' pages as fp16 planes

Query i and key j are positions in one document (or request). A score is s = scale * q . k, capped to
cap * tanh(s / cap) where cap > 0, less slope[head] * |i - j| where the case has a bias; with win > 0 a query sees the
keys j <= i that are sinks (j < sink) or recent (j > i - win), else all j <= i, and every key of its document's prefix.

Pages hold 16-row groups of one kv head, a K part and a V part of 9 * head_dim + 32 bytes each: codes,
block scales (binary16) and row factors (bfloat16 powers of two); include/fa.h gives the byte order.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}


# ----------------------------------------------------------------- the cases

def listed():
    return [
        # a few short answers, one forward call: latency
        {"name": "packed_short", "kind": "packed", "dtype": "bf16", "docs": 3, "tokens": 203, "hq": 8, "hkv": 2, "hd": 64,
         "cap": 0.0, "bias": False, "prefix": 0, "sink": 0, "win": 0},
        # a batch of documents of every length, capped scores, the heads that the benchmark times
        {"name": "packed_docs", "kind": "packed", "dtype": "bf16", "docs": 23, "tokens": 8192, "hq": 16, "hkv": 2,
         "hd": 256, "cap": 30.0, "bias": False, "prefix": 0, "sink": 0, "win": 0},
        # one long document, scores that fall with the distance
        {"name": "packed_long", "kind": "packed", "dtype": "f16", "docs": 1, "tokens": 16384, "hq": 8, "hkv": 8, "hd": 128,
         "cap": 0.0, "bias": True, "prefix": 0, "sink": 0, "win": 0},
        # prompts whose first part sees itself whole, then a window
        {"name": "packed_prefix", "kind": "packed", "dtype": "bf16", "docs": 5, "tokens": 11003, "hq": 16, "hkv": 4,
         "hd": 128, "cap": 0.0, "bias": False, "prefix": 700, "sink": 4, "win": 1024},
        # the gradient of a few short answers
        {"name": "grad_short", "kind": "grad", "dtype": "f16", "docs": 4, "tokens": 301, "hq": 4, "hkv": 4, "hd": 64,
         "cap": 0.0, "bias": True, "prefix": 0, "sink": 0, "win": 0},
        # of the documents above, capped scores, wide heads
        {"name": "grad_docs", "kind": "grad", "dtype": "bf16", "docs": 23, "tokens": 8192, "hq": 16, "hkv": 2, "hd": 256,
         "cap": 30.0, "bias": False, "prefix": 0, "sink": 0, "win": 0},
        # of one long document
        {"name": "grad_long", "kind": "grad", "dtype": "bf16", "docs": 1, "tokens": 16384, "hq": 8, "hkv": 2, "hd": 128,
         "cap": 0.0, "bias": False, "prefix": 0, "sink": 0, "win": 0},
        # of prompts with a prefix and a window, narrow heads
        {"name": "grad_prefix", "kind": "grad", "dtype": "f16", "docs": 9, "tokens": 10007, "hq": 16, "hkv": 8, "hd": 64,
         "cap": 20.0, "bias": False, "prefix": 300, "sink": 4, "win": 1024},
        # one short request, capped scores: latency alone
        {"name": "paged_one", "kind": "paged", "dtype": "f16", "reqs": 1, "rows": 600, "ragged": False, "nq": 1, "hq": 8,
         "hkv": 2, "hd": 64, "page_rows": 16, "cap": 30.0, "bias": False, "sink": 0, "win": 0},
        # a decode step of 48 requests of every length, capped scores that fall with the distance
        {"name": "paged_ragged", "kind": "paged", "dtype": "bf16", "reqs": 48, "rows": 30000, "ragged": True, "nq": 1,
         "hq": 32, "hkv": 8, "hd": 128, "page_rows": 32, "cap": 50.0, "bias": True, "sink": 0, "win": 0},
        # speculative decoding's few rows over short caches
        {"name": "append_rows", "kind": "append", "dtype": "f32", "reqs": 8, "cached": 29, "fresh": 3, "hq": 8, "hkv": 2,
         "hd": 64, "rd": 64, "axes": 1, "adjacent": False, "page_rows": 16},
        # chunks of several prompts
        {"name": "append_prompt", "kind": "append", "dtype": "bf16", "reqs": 6, "cached": 11, "fresh": 5000, "hq": 16,
         "hkv": 4, "hd": 128, "rd": 128, "axes": 1, "adjacent": False, "page_rows": 64},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["packed", "packed", "grad", "grad", "paged", "append"])
    hd = rng.choice([64, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    page_rows = rng.choice([16, 32, 64, 128, 256])
    sink, win = rng.choice([(0, 0), (0, 0), (4, 1024), (0, 333), (37, 61)])
    cap, bias = rng.choice([0.0, 20.0, 50.0]), rng.random() < 0.4
    if kind in ("packed", "grad"):
        hq = hkv * rng.choice([g for g in (1, 2, 4, 8, 16) if g * hkv <= 32])
        # no more pairs of a query and a key than the longest listed ones have, all heads together
        tokens = _log(rng, 1, int(math.sqrt((1 << 31) / max(hq, 8) * min(1.0, 128 / hd))))
        docs = _log(rng, 1, max(1, min(200, tokens // 3)))
        return {"kind": kind, "dtype": rng.choice(["f16", "bf16"]), "docs": docs, "tokens": tokens, "hq": hq, "hkv": hkv,
                "hd": hd, "cap": cap, "bias": bias, "prefix": rng.choice([0, 0, 1, _log(rng, 2, 1000)]), "sink": sink,
                "win": win}
    dtype = rng.choice(["f32", "f16", "bf16"])
    hq = hkv * rng.choice([1, 2, 4, 8, 16])
    if kind == "append":
        axes = rng.choice([1, 1, 2, 3])
        most = 30000 * 4 * 128 // (hkv * hd)  # rows, so that no case costs more than the largest listed one
        most = min(most, 30000 * 20 * 128 // ((hq + hkv) * hd))
        reqs = _log(rng, 1, 64)
        rows = _log(rng, 2, max(2, most // reqs))
        fresh = _log(rng, 1, rows)
        return {"kind": kind, "dtype": dtype, "reqs": reqs, "cached": rows - fresh, "fresh": fresh, "hq": hq, "hkv": hkv,
                "hd": hd, "rd": rng.choice([hd, hd // 2, 64]), "axes": axes, "adjacent": rng.random() < 0.5,
                "page_rows": page_rows}
    rows = _log(rng, 1, 30000)
    most = 12 * 30000 * 1024 // (hkv * hd * rows)
    nq = rng.choice([1, 1, 1, 2, 5])
    reqs = _log(rng, 1, max(1, min(256, most // (2 * max(1, hq // hkv * nq // 8)))))
    return {"kind": kind, "dtype": dtype, "reqs": reqs, "rows": rows, "ragged": rng.random() < 0.7, "nq": nq, "hq": hq,
            "hkv": hkv, "hd": hd, "page_rows": page_rows, "cap": cap or 30.0, "bias": bias, "sink": sink, "win": win}


# ------------------------------------------------- lengths that a case stands for

def _spread(n, top, floor=0):
    """n lengths up to `top`, even in their logarithm, from one row up; every seventh of many is `floor`."""
    i = np.arange(n)
    v = np.maximum(1, np.rint(np.exp(np.log(max(top, 1)) * (i + 1) / n))).astype(np.int64)
    return np.where((i % 7 == 3) & (n >= 8), floor, v)


def _attn_lengths(c):
    if not c["ragged"]:
        rows = np.full(c["reqs"], c["rows"])
        return rows, np.minimum(c["nq"], rows)
    rows = _spread(c["reqs"], c["rows"])
    return rows, np.minimum(1 + np.arange(c["reqs"]) % c["nq"], np.maximum(rows, 1))


def _chunk_lengths(c):
    i = np.arange(c["reqs"])
    return np.maximum(0, c["cached"] - 5 * i), np.maximum(1, c["fresh"] - 3 * i)


def _doc_lengths(c):
    """Lengths of the documents, of `tokens` in all, spread in their logarithm; each seventh of many is empty."""
    n = c["docs"]
    share = np.where((np.arange(n) % 7 == 3) & (n >= 8), 0.0, np.exp(3.5 * (np.arange(n) + 1) / n))
    edge = np.rint(np.cumsum(share) / share.sum() * c["tokens"]).astype(np.int64)
    return np.diff(edge, prepend=0)


def _pairs(n, prefix, sink, win):
    """Pairs of a query and a key that it sees in a document of n tokens."""
    i = np.arange(int(n))
    first = np.minimum(prefix, n)
    lo = np.maximum(0, i - win + 1) if win > 0 else np.zeros_like(i)
    head = np.maximum(first, np.minimum(sink, i + 1) if win > 0 else 0)  # seen from the document's start
    return int((np.minimum(head, np.maximum(lo, first)) + np.maximum(0, i + 1 - np.maximum(lo, first))).sum())


def _visible(rows, nq, sink, win):
    """Rows of a request that any of its queries attends."""
    if win <= 0:
        return rows
    lo = np.maximum(0, rows - nq - win + 1)
    return np.where(rows > 0, np.minimum(lo, sink) + rows - lo, 0)


def work(case):
    c = case
    size = BYTES[c["dtype"]]
    if c["kind"] in ("packed", "grad"):
        pairs = sum(_pairs(n, c["prefix"], c["sink"], c["win"]) for n in _doc_lengths(c))
        q, kv = c["tokens"] * c["hq"] * c["hd"] * size, c["tokens"] * c["hkv"] * c["hd"] * size
        lse = 4 * c["tokens"] * c["hq"]
        # products: q . k and p v; in the gradient q . k, dout . v, and those of dq, dk, dv
        if c["kind"] == "packed":
            return {"bytes": 2 * q + 2 * kv + lse, "flops": 4 * pairs * c["hq"] * c["hd"]}
        return {"bytes": 4 * q + 4 * kv + lse, "flops": 10 * pairs * c["hq"] * c["hd"]}
    if c["kind"] == "append":
        cached, fresh = _chunk_lengths(c)
        row = c["hkv"] * (18 * c["hd"] + 64) // 16
        new, rows = int(fresh.sum()), int((cached + fresh).sum())
        return {"bytes": new * (2 * c["hq"] + 2 * c["hkv"]) * c["hd"] * size + 4 * new * (1 + c["axes"]) + (new + rows) * row
                + rows * c["hkv"] * c["hd"] * 4, "flops": 3 * new * (c["hq"] + c["hkv"]) * c["rd"]}
    rows, nq = _attn_lengths(c)
    seen = _visible(rows, nq, c["sink"], c["win"])
    return {"bytes": int(seen.sum() * c["hkv"] * (18 * c["hd"] + 64) // 16
                         + nq.sum() * c["hq"] * (2 * c["hd"] * size + 4)),
            "flops": int((seen * nq).sum() * c["hq"] * c["hd"] * 4)}


# ------------------------------------------------------------------- inputs

def _int(a, device="cuda"):
    return torch.as_tensor(np.ascontiguousarray(a), dtype=torch.int32, device=device)


def _quantise(x):
    """4-bit rows of x [..., head_dim] fp32: codes 0..15 [..., hd], block scales binary16 [..., hd / 32] and
    the rows' power-of-two factors [...], in the steps of the Q4_0 encoder."""
    xb = x.unflatten(-1, (-1, 32))
    d = xb.abs().amax(-1) / -8
    inv = torch.where(d != 0, 1 / d, 0.0)
    codes = (torch.round(xb * inv.unsqueeze(-1)) + 8).clamp(0, 15).to(torch.uint8).flatten(-2)
    top = d.abs().amax(-1)
    factor = torch.where(top > 0, torch.exp2(torch.frexp(top)[1].float() - 1), 1.0)
    return codes, (d / factor.unsqueeze(-1)).half(), factor


def _pack_part(codes, scales, factors, v):
    """One part (K, or V) of 16-row groups: codes [..., 16, hd] -> bytes [..., 9 hd + 32]."""
    hd, lead = codes.shape[-1], codes.shape[:-2]
    nb, k = hd // 32, len(lead)
    ax = lambda *a: [*range(k), *[k + i for i in a]]  # noqa: E731
    if not v:
        c = codes.reshape(*lead, 2, 8, nb, 4, 8).permute(ax(0, 2, 1, 3, 4))   # half, block, g, t, 8
        c = c.reshape(*lead, nb // 2, 4, 8, 4, 8).permute(ax(0, 2, 3, 1, 4))  # chunk, g, t, word, 8
        s = scales
    else:
        c = codes.reshape(*lead, 2, 4, 2, nb, 8, 4).permute(ax(0, 2, 3, 4, 1, 5))  # half, low, block, g, t, 4
        c = c.reshape(*lead, nb // 2, 8, 8, 4, 4).permute(ax(0, 2, 3, 1, 4))       # chunk, g, t, half word, 4
        s = scales.reshape(*lead, 2, 4, 2, nb // 2, 2).permute(ax(3, 1, 4, 0, 2))   # block pair, t, block, half, low
    c = c.reshape(*lead, 8 * hd, 2)
    c = c[..., 0] | c[..., 1] << 4
    return torch.cat([c, s.reshape(*lead, 16 * nb).contiguous().view(torch.uint8),
                      factors.bfloat16().contiguous().view(torch.uint8)], -1)


def _unpack_part(part, hd, v):
    """Bytes [..., 9 hd + 32] -> the values [..., 16, hd] they stand for, fp32."""
    lead, nb = part.shape[:-1], hd // 32
    k = len(lead)
    ax = lambda *a: [*range(k), *[k + i for i in a]]  # noqa: E731
    c = part[..., :8 * hd]
    c = torch.stack([c & 15, c >> 4], -1)
    s = part[..., 8 * hd:9 * hd].contiguous().view(torch.float16)
    f = part[..., 9 * hd:].contiguous().view(torch.bfloat16).float()
    if not v:
        c = c.reshape(*lead, nb // 2, 8, 4, 4, 8).permute(ax(0, 3, 1, 2, 4))
        c = c.reshape(*lead, 2, nb, 8, 4, 8).permute(ax(0, 2, 1, 3, 4))
        s = s.reshape(*lead, 16, nb)
    else:
        c = c.reshape(*lead, nb // 2, 8, 4, 8, 4).permute(ax(0, 3, 1, 2, 4))
        c = c.reshape(*lead, 2, 2, nb, 8, 4, 4).permute(ax(0, 4, 1, 2, 3, 5))
        s = s.reshape(*lead, nb // 2, 4, 2, 2, 2).permute(ax(3, 1, 4, 0, 2)).reshape(*lead, 16, nb)
    c = c.reshape(*lead, 16, nb, 32).float() - 8
    return (c * (s.float() * f.unsqueeze(-1)).unsqueeze(-1)).flatten(-2)


def _pool(g, n_pages, hkv, page_rows, hd):
    """Pages whose rows are quantised N(0, 1) values with a few strong channels in K."""
    shape = (n_pages, hkv, page_rows // 16, 16, hd)
    strong = 1 + 3 * (torch.rand(hkv, 1, 1, hd, device="cuda", generator=g) < 0.02)
    k = torch.randn(shape, device="cuda", generator=g) * strong
    parts = [_pack_part(*_quantise(k), False)]
    k.normal_(generator=g)
    parts.append(_pack_part(*_quantise(k), True))
    return torch.cat(parts, -1).flatten()


def _table(rng, rows, page_rows):
    """A block table over pages in random order, one page in each eight free; entries past a request's rows: -1."""
    pages = -(-rows // page_rows)
    n = max(1, int(pages.sum() * 8 // 7) + 1)
    order, table = rng.permutation(n), np.full((len(rows), max(1, int(pages.max()))), -1, np.int64)
    table[np.arange(table.shape[1]) < pages[:, None]] = order[:pages.sum()]
    return table, n


def _slopes(c):
    """Powers of two that fall from head to head, or None."""
    if not c["bias"]:
        return None
    return torch.exp2(-8.0 * (torch.arange(c["hq"], device="cuda") + 1) / c["hq"]).float()


def prepare(case, seed):
    c = case
    rng = np.random.default_rng(seed)
    g = torch.Generator("cuda").manual_seed(seed)
    s = dict(c)
    dt = DTYPES[c["dtype"]]
    rand = lambda *shape: torch.randn(shape, device="cuda", generator=g).to(dt)  # noqa: E731
    if c["kind"] in ("packed", "grad"):
        hq, hkv, hd, n = c["hq"], c["hkv"], c["hd"], c["tokens"]
        lens = rng.permutation(_doc_lengths(c))
        T = n + 5  # the batch is padded: 5 tokens of no document
        qkv = rand(T, hq + 2 * hkv, hd)  # one projection's output
        if c["cap"]:
            qkv[:, :hq] *= 4  # scores that the cap is there for
        cu = np.concatenate([[0], np.cumsum(lens)])
        # a document and a position for each token; the padding's: a document of its own
        doc = np.repeat(np.arange(c["docs"]), lens)
        pos = np.arange(n) - cu[doc]
        zeros = lambda heads: torch.zeros(T, heads, hd, dtype=dt, device="cuda")  # noqa: E731
        s.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], cu=_int(cu),
                 prefixes=_int(np.minimum(c["prefix"], lens)) if c["prefix"] else None, slopes=_slopes(c),
                 doc=torch.as_tensor(doc, device="cuda"), pos=torch.as_tensor(pos, device="cuda"), out=zeros(hq),
                 lse=torch.zeros(hq, T, device="cuda"),
                 # scratch: what fa.packed_attn_workspace_bytes and its gradient's ask for is below this
                 workspace=torch.empty((64 << 20) + 32 * hq * T + 4096 * hkv * c["docs"], dtype=torch.uint8, device="cuda"))
        if c["kind"] == "grad":
            made = _plain_packed(s)
            s.update(out=made["out"], lse=made["lse"], dout=0.02 * rand(T, hq, hd), dq=zeros(hq), dk=zeros(hkv), dv=zeros(hkv))
        return s
    if c["kind"] == "append":
        cached, fresh = _chunk_lengths(c)
        rows = cached + fresh
        table, n = _table(rng, rows, c["page_rows"])
        T, A, half = int(fresh.sum()), c["axes"], c["rd"] // 2
        req = np.repeat(np.arange(c["reqs"]), fresh)
        at = np.arange(T) - np.repeat(np.cumsum(fresh) - fresh, fresh) + cached[req]
        slots = table[req, at // c["page_rows"]] * c["page_rows"] + at % c["page_rows"]
        pos = rng.integers(0, 4096, (A, T))
        pos[0] = at + rng.integers(0, 1 << 17)
        axis = np.arange(half) % A
        inv_freq = 1e6 ** (-np.arange(half) / half)
        max_seq = int(rows.max()) + 3
        plane = (c["hkv"] * max_seq * c["hd"] * 2 + 255) // 256 * 256
        qkv = rand(T, c["hq"] + 2 * c["hkv"], c["hd"])
        s.update(pages=_pool(g, n, c["hkv"], c["page_rows"], c["hd"]), table=_int(table), lens=_int(rows), slots=_int(slots),
                 req=torch.as_tensor(req, device="cuda"), at=torch.as_tensor(at, device="cuda"), q=qkv[:, :c["hq"]],
                 k=qkv[:, c["hq"]:c["hq"] + c["hkv"]], v=qkv[:, c["hq"] + c["hkv"]:], pos=_int(pos), max_seq=max_seq,
                 axis=torch.as_tensor(axis, device="cuda"),
                 inv_freq=torch.tensor(inv_freq, dtype=torch.float64, device="cuda"),
                 # what fa.rope_table makes once for a model: each pair's turns per position and its axis
                 rope=_turns(inv_freq, axis), q_out=torch.empty(T, c["hq"], c["hd"], dtype=dt, device="cuda"),
                 k_planes=torch.zeros(c["reqs"] * plane, dtype=torch.uint8, device="cuda"),
                 v_planes=torch.zeros(c["reqs"] * plane, dtype=torch.uint8, device="cuda"))
        return s
    rows, nq = _attn_lengths(c)
    mix = rng.permutation(c["reqs"])
    rows, nq = rows[mix], nq[mix]
    table, n = _table(rng, rows, c["page_rows"])
    T = int(nq.sum())
    s.update(pages=_pool(g, n, c["hkv"], c["page_rows"], c["hd"]), table=_int(table), lens=_int(rows),
             cu=_int(np.concatenate([[0], np.cumsum(nq)])), q=4 * rand(T, c["hq"], c["hd"]), n_q=int(nq.max()),
             req=torch.as_tensor(np.repeat(np.arange(c["reqs"]), nq), device="cuda"), slopes=_slopes(c),
             out=torch.empty(T, c["hq"], c["hd"], dtype=dt, device="cuda"),
             lse=torch.empty(c["hq"], T, device="cuda"),
             workspace=torch.empty(64 << 20, dtype=torch.uint8, device="cuda"))
    return s


def _turns(inv_freq, axis):
    """[pairs][4] int32: low and high word of 2^64 * (inv_freq / 2 pi), the axis, 0."""
    turns = [int(math.floor(math.ldexp(f / (2 * math.pi) % 1.0, 64))) for f in inv_freq]
    t = np.array([[x & 0xffffffff, x >> 32, int(a), 0] for x, a in zip(turns, axis)], np.uint32)
    return torch.as_tensor(t.view(np.int32), device="cuda")


# ---------------------------------------------------------------- one pass

def run(state):
    s = state
    return {"packed": _run_packed, "grad": _run_grad, "paged": _run_paged, "append": _run_append}[s["kind"]](s)


def _run_packed(s):
    if own:
        import causal_gqa_flash_attn_gb300 as fa
        fa.packed_attn(s["q"], s["k"], s["v"], s["out"], s["cu"], prefix=s["prefixes"], sink=s["sink"], win=s["win"],
                       cap=s["cap"], slopes=s["slopes"], lse=s["lse"], workspace=s["workspace"])
        return {"out": s["out"], "lse": s["lse"]}
    return _plain_packed(s)


def _scores(s, q, k):
    """[hkv][group][n][n] scores, -inf where a query does not see a key, and the factor of the cap's derivative."""
    n, hd = q.shape[-2:]
    x = (q.flatten(1, 2) @ k.transpose(-1, -2)).view(*q.shape[:3], n) / math.sqrt(hd)
    slope = 1.0
    if s["cap"]:
        x = torch.tanh(x / s["cap"])
        slope = 1 - x * x
        x = x * s["cap"]
    i, j = s["pos"].unsqueeze(1), s["pos"].unsqueeze(0)
    if s["slopes"] is not None:
        x = x - s["slopes"].view(q.shape[0], -1, 1, 1) * (i - j).abs()
    see = j <= i
    if s["win"] > 0:
        see &= (j < s["sink"]) | (j > i - s["win"])
    if s["prefixes"] is not None:
        see |= j < s["prefixes"].long()[s["doc"]].unsqueeze(0)
    see &= s["doc"].unsqueeze(1) == s["doc"].unsqueeze(0)
    return torch.where(see, x, -math.inf), slope


def _by_head(x, hkv, n):
    """[tokens][heads][hd] -> the first n tokens as [hkv][group][n][hd] fp32."""
    return x[:n].float().unflatten(1, (hkv, -1)).permute(1, 2, 0, 3)


def _by_token(x, like):
    """[hkv][group][n][hd] -> [tokens][heads][hd] in the type of `like`; zeros for the padding."""
    x = x.permute(2, 0, 1, 3).flatten(1, 2).to(like.dtype)
    return torch.cat([x, x.new_zeros(like.shape[0] - x.shape[0], *x.shape[1:])])


def _plain_packed(s):
    n, hkv = s["tokens"], s["hkv"]
    q, k, v = (_by_head(s[name], hkv, n) for name in "qkv")
    score, _ = _scores(s, q, k[:, 0])
    top = score.amax(-1, keepdim=True)
    w = torch.exp(score - top)
    total = w.sum(-1, keepdim=True)
    out = ((w / total).flatten(1, 2) @ v[:, 0]).view(q.shape)
    lse = (top + total.log()).squeeze(-1).flatten(0, 1)
    return {"out": _by_token(out, s["q"]), "lse": torch.cat([lse, lse.new_zeros(s["hq"], s["q"].shape[0] - n)], 1)}


def _run_grad(s):
    if own:
        import causal_gqa_flash_attn_gb300 as fa
        fa.packed_attn_grad(s["q"], s["k"], s["v"], s["out"], s["lse"], s["dout"], s["dq"], s["dk"], s["dv"], s["cu"],
                            prefix=s["prefixes"], sink=s["sink"], win=s["win"], cap=s["cap"], slopes=s["slopes"],
                            workspace=s["workspace"])
        return {"dq": s["dq"], "dk": s["dk"], "dv": s["dv"]}
    n, hkv = s["tokens"], s["hkv"]
    q, k, v, out, dout = (_by_head(s[name], hkv, n) for name in ("q", "k", "v", "out", "dout"))
    score, slope = _scores(s, q, k[:, 0])
    w = torch.exp(score - s["lse"][:, :n].view(hkv, -1, n, 1)).flatten(1, 2)  # [hkv][group * n][n]
    dv = w.transpose(-1, -2) @ dout.flatten(1, 2)
    dw = dout.flatten(1, 2) @ v[:, 0].transpose(-1, -2)
    ds = w * (dw - (out * dout).sum(-1).flatten(1, 2).unsqueeze(-1)) / math.sqrt(s["hd"])
    if s["cap"]:
        ds = ds * slope.flatten(1, 2)
    dq = (ds @ k[:, 0]).view(q.shape)
    dk = ds.transpose(-1, -2) @ q.flatten(1, 2)
    return {"dq": _by_token(dq, s["q"]), "dk": _by_token(dk.unsqueeze(1), s["k"]), "dv": _by_token(dv.unsqueeze(1), s["v"])}


def _turn(s, x):
    """The rotated x [tokens][heads][hd], rounded to its type."""
    angle = s["pos"].double()[s["axis"]].T * s["inv_freq"]  # [tokens][pairs]; 64 bits: far positions
    cos, sin, rd = angle.cos().float().unsqueeze(1), angle.sin().float().unsqueeze(1), s["rd"]
    y = x.float()
    r = y[..., :rd].unflatten(-1, (-1, 2)).transpose(-1, -2) if s["adjacent"] else y[..., :rd].unflatten(-1, (2, -1))
    a, b = r[..., 0, :], r[..., 1, :]
    r = torch.stack([a * cos - b * sin, a * sin + b * cos], -2)
    r = (r.transpose(-1, -2) if s["adjacent"] else r).flatten(-2)
    return torch.cat([r, y[..., rd:]], -1).to(x.dtype)


def _planes(s):
    """The fp16 planes [requests][hkv][max_seq][hd] as the values they hold."""
    n, rows = s["reqs"], s["hkv"] * s["max_seq"] * s["hd"]
    cut = lambda p: p.view(n, -1)[:, :2 * rows].view(torch.float16).view(n, s["hkv"], s["max_seq"], s["hd"])  # noqa: E731
    return {"k": cut(s["k_planes"]), "v": cut(s["v_planes"])}


def _rows_of(s):
    """K and V of the requests' pages [requests][hkv][rows][hd] fp32; rows of no page are some page's."""
    P, hd = s["page_rows"], s["hd"]
    atoms = s["pages"].view(-1, s["hkv"], P // 16, 18 * hd + 64)
    atoms = atoms[s["table"].long().clamp(min=0)].transpose(1, 2)  # [requests][hkv][pages][groups][bytes]
    k, v = atoms.split(9 * hd + 32, -1)
    return _unpack_part(k, hd, False).flatten(2, 4), _unpack_part(v, hd, True).flatten(2, 4)


def _run_append(s):
    if own:
        import causal_gqa_flash_attn_gb300 as fa
        fa.rope_append(s["q"], s["k"], s["v"], s["q_out"], s["pos"], s["rope"], s["slots"], s["pages"],
                       page_rows=s["page_rows"], adjacent=s["adjacent"])
        fa.paged_gather(s["pages"], s["table"], s["lens"], s["k_planes"], s["v_planes"], n_kv_heads=s["hkv"],
                        head_dim=s["hd"], page_rows=s["page_rows"], max_seq=s["max_seq"])
        return {"q": s["q_out"], **_planes(s)}
    k, v = _rows_of(s)
    live = (torch.arange(s["max_seq"], device="cuda") < s["lens"].unsqueeze(1))[:, None, :, None]
    # the pages hold the 4-bit codes of k as rotated in its own type
    return {"q": _turn(s, s["q"]), "k": _plane(s, k, _turn(s, s["k"]), live), "v": _plane(s, v, s["v"], live)}


def _plane(s, old, new, live):
    """The rows of the pages `old` with those that the codes of `new` stand for, [requests][hkv][max_seq][hd]."""
    codes, scales, factors = _quantise(new.float())
    x = (codes.float() - 8).unflatten(-1, (-1, 32)) * (scales.float() * factors.unsqueeze(-1)).unsqueeze(-1)
    plane = torch.zeros(live.shape[0], s["hkv"], s["max_seq"], s["hd"], device="cuda")
    n = min(s["max_seq"], old.shape[2])
    plane[:, :, :n] = old[:, :, :n]
    plane[s["req"], :, s["at"]] = x.flatten(-2)
    return torch.where(live, plane, 0.0).half()


def _run_paged(s):
    if own:
        import causal_gqa_flash_attn_gb300 as fa
        fa.paged_attn(s["q"], s["out"], s["cu"], s["lens"], s["table"], s["pages"], n_kv_heads=s["hkv"],
                      page_rows=s["page_rows"], sink=s["sink"], win=s["win"], cap=s["cap"], slopes=s["slopes"],
                      lse=s["lse"], workspace=s["workspace"])
        return {"out": s["out"], "lse": s["lse"]}
    k, v = _rows_of(s)
    R, hkv, rows, hd = k.shape
    cu, lens = s["cu"].long(), s["lens"].long()
    nth = torch.arange(s["req"].numel(), device="cuda") - cu[s["req"]]  # a token's place in its request
    q = torch.zeros(R, s["n_q"], s["hq"], hd, device="cuda")
    q[s["req"], nth] = s["q"].float()
    q = q.view(R, s["n_q"], hkv, -1, hd).permute(0, 2, 1, 3, 4)  # [requests][hkv][queries][group][hd]
    score = (q.flatten(2, 3) @ k.transpose(-1, -2)) / math.sqrt(hd)
    score = s["cap"] * torch.tanh(score / s["cap"])
    score = score.view(R, hkv, s["n_q"], -1, rows)
    j = torch.arange(rows, device="cuda")
    p = (lens - (cu[1:] - cu[:-1])).unsqueeze(1) + torch.arange(s["n_q"], device="cuda")
    p = p[:, None, :, None, None]
    if s["slopes"] is not None:
        score = score - s["slopes"].view(hkv, 1, -1, 1) * (p - j).abs()
    see = j <= p
    if s["win"] > 0:
        see &= (j < s["sink"]) | (j > p - s["win"])
    score = torch.where(see, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    w = torch.exp(score - torch.where(top > -math.inf, top, 0.0))
    total = w.sum(-1, keepdim=True)
    w = w / torch.where(total > 0, total, 1.0)
    out = (w.flatten(2, 3) @ v).view(R, hkv, s["n_q"], -1, hd).permute(0, 2, 1, 3, 4).flatten(2, 3)
    lse = (top + total.log()).squeeze(-1).permute(0, 2, 1, 3).flatten(2, 3)
    return {"out": out[s["req"], nth].to(s["q"].dtype), "lse": lse[s["req"], nth].T.contiguous()}


# ------------------------------------------------ the definition, in 64 bits

def _places(hd, v):
    """Where element e of row r of a part lies: byte [16][hd] and shift of its code, byte of its scale."""
    nb = hd // 32
    r, e = np.arange(16)[:, None], np.arange(hd)[None, :]
    b = e // 32
    if not v:
        j = r // 8 * nb + b
        word = (j // 4 * 32 + r % 8 * 4 + e % 32 // 8) * 4 + j % 4
        at, shift, scale = word * 4 + e % 8 // 2, e % 2 * 4, 8 * hd + 2 * (r * nb + b)
    else:
        t, x = r % 8 // 2, r % 2 + 2 * (r // 8)
        j = x * nb + b
        word = (j // 8 * 32 + e % 32 // 4 * 4 + t) * 8 + j % 8
        at, shift, scale = word * 2 + e % 4 // 2, e % 2 * 4, 8 * hd + 2 * ((b // 2 * 4 + t) * 8 + b % 2 * 4 + x)
    return [torch.as_tensor(np.broadcast_to(a, (16, hd)).copy(), device="cuda") for a in (at, shift, scale)]


def _value(part, hd, v):
    """[n][9 hd + 32] bytes -> [16 n][hd] values in 64 bits, element by element."""
    at, shift, scale = _places(hd, v)
    code = (part[:, at].int() >> shift) & 15
    bits = part[:, scale].int() | part[:, scale + 1].int() << 8
    sign, ex, man = bits >> 15, (bits >> 10) & 31, (bits & 1023).double()
    size = torch.where(ex > 0, (1024 + man) * torch.exp2(ex.double() - 25), man * 2.0 ** -24) * (1 - 2 * sign)
    fa = 9 * hd + 2 * torch.arange(16, device="cuda")
    factor = torch.exp2(((part[:, fa].int() | part[:, fa + 1].int() << 8) >> 7).double() - 127)
    return ((code - 8).double() * size * factor.unsqueeze(-1)).flatten(0, 1)


def _request(s, r, first, last):
    """Rows [first, last) of request r: K and V [hkv][rows][hd] in 64 bits."""
    P, hd, hkv = s["page_rows"], s["hd"], s["hkv"]
    size = 18 * hd + 64
    g = torch.arange(first // 16, -(-last // 16), device="cuda")
    page = s["table"][r].long()[g // (P // 16)]
    k, v = [], []
    for h in range(hkv):
        start = ((page * hkv + h) * (P // 16) + g % (P // 16)) * size
        atom = s["pages"][start.unsqueeze(1) + torch.arange(size, device="cuda")]
        skip, n = first - first // 16 * 16, last - first
        k.append(_value(atom[:, :size // 2], hd, False)[skip:skip + n])
        v.append(_value(atom[:, size // 2:], hd, True)[skip:skip + n])
    return torch.stack(k), torch.stack(v)


def _exact_append(c, s):
    made = {}
    rd = c["rd"]
    angle = torch.stack([s["pos"][a].double() * f for a, f in zip(s["axis"].tolist(), s["inv_freq"].tolist())], 1)
    z = torch.polar(torch.ones_like(angle), angle).unsqueeze(1)
    i = torch.arange(rd // 2, device="cuda")
    re, im = (2 * i, 2 * i + 1) if c["adjacent"] else (i, i + rd // 2)
    for name in ("q", "k"):
        x = s[name].double().clone()
        y = torch.complex(x[..., re], x[..., im]) * z
        x[..., re], x[..., im] = y.real, y.imag
        made[name] = x
    new = {"k": made["k"].to(s["k"].dtype), "v": s["v"]}
    cached, fresh = _chunk_lengths(c)
    plane = {n: torch.zeros(c["reqs"], c["hkv"], s["max_seq"], c["hd"], dtype=torch.float64, device="cuda") for n in "kv"}
    t = 0
    for r in range(c["reqs"]):
        if cached[r]:
            plane["k"][r, :, :cached[r]], plane["v"][r, :, :cached[r]] = _request(s, r, 0, int(cached[r]))
        for n in "kv":
            x = new[n][t:t + fresh[r]].float().cpu().numpy().reshape(int(fresh[r]), c["hkv"], -1, 32)
            d = (np.abs(x).max(-1) / np.float32(-8)).astype(np.float32)
            inv = np.divide(np.float32(1), d, out=np.zeros_like(d), where=d != 0)
            code = np.clip(np.rint(x * inv[..., None]) + 8, 0, 15)
            top = np.abs(d).max(-1).astype(np.float64)
            e = np.floor(np.log2(np.where(top > 0, top, 1.0)))
            scale = (d.astype(np.float64) * 2.0 ** -e[..., None]).astype(np.float16).astype(np.float64) * 2.0 ** e[..., None]
            rows = torch.as_tensor((code - 8) * scale[..., None]).flatten(-2).transpose(0, 1)
            plane[n][r, :, cached[r]:cached[r] + fresh[r]] = rows.cuda()
        t += int(fresh[r])
    return {"q": made["q"], **plane}


def _softmax(c, x, i, j, prefix, slope):
    """Weights, log-sum-exp and the cap's derivative of scores x [..., i, j] in 64 bits; slope [..., 1, 1] or None."""
    down = torch.ones_like(x)
    if c["cap"]:
        down = 1 / torch.cosh(x / c["cap"]) ** 2
        x = c["cap"] * torch.tanh(x / c["cap"])
    far = i[:, None] - j
    if slope is not None:
        x = x - slope.double() * far.abs()
    hide = far < 0
    if c["win"] > 0:
        hide |= (far >= c["win"]) & (j >= c["sink"])
    hide &= j >= prefix
    x = x.masked_fill(hide, -math.inf)
    lse = torch.logsumexp(x, -1)
    return torch.exp(x - lse.unsqueeze(-1)), lse, down


def _exact_packed(c, s):
    hd, group = c["hd"], c["hq"] // c["hkv"]
    wide = lambda x: torch.zeros(x.shape, dtype=torch.float64, device="cuda")  # noqa: E731
    out, lse, dq, dk, dv = (wide(s[n]) for n in ("q", "q", "q", "k", "v"))
    lse = torch.zeros(c["hq"], out.shape[0], dtype=torch.float64, device="cuda")
    cu = s["cu"].tolist()
    for d in range(c["docs"]):
        at = slice(cu[d], cu[d + 1])
        n = cu[d + 1] - cu[d]
        if not n:
            continue
        prefix = 0 if s["prefixes"] is None else int(s["prefixes"][d])
        i = torch.arange(n, device="cuda")
        for h in range(c["hq"]):
            q, k, v = s["q"][at, h].double(), s["k"][at, h // group].double(), s["v"][at, h // group].double()
            slope = None if s["slopes"] is None else s["slopes"][h]
            p, z, down = _softmax(c, q @ k.T / math.sqrt(hd), i, i, prefix, slope)
            out[at, h], lse[h, at] = p @ v, z
            if c["kind"] == "grad":
                do = s["dout"][at, h].double()
                dp = do @ v.T
                dx = p * (dp - (p * dp).sum(-1, keepdim=True)) * down / math.sqrt(hd)
                dq[at, h] = dx @ k
                dk[at, h // group] += dx.T @ q
                dv[at, h // group] += p.T @ do
    return {"dq": dq, "dk": dk, "dv": dv} if c["kind"] == "grad" else {"out": out, "lse": lse}


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["kind"] == "append":
        return _exact_append(c, s)
    if c["kind"] in ("packed", "grad"):
        return _exact_packed(c, s)
    lens, cu = s["lens"].tolist(), s["cu"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full((c["hq"], s["q"].shape[0]), -math.inf, dtype=torch.float64, device="cuda")
    slope = None if s["slopes"] is None else s["slopes"].view(-1, 1, 1)
    for r in range(c["reqs"]):
        if not lens[r]:
            continue
        k, v = _request(s, r, 0, lens[r])
        k, v = (x.repeat_interleave(c["hq"] // c["hkv"], 0) for x in (k, v))
        at = slice(cu[r], cu[r + 1])
        i = lens[r] - cu[r + 1] + torch.arange(cu[r], cu[r + 1], device="cuda")
        x = torch.einsum("qhd,hjd->hqj", s["q"][at].double(), k) / math.sqrt(c["hd"])
        p, lse[:, at], _ = _softmax(c, x, i, torch.arange(lens[r], device="cuda"), 0, slope)
        out[at] = torch.einsum("hqj,hjd->qhd", p, v)
    return {"out": out, "lse": lse}
