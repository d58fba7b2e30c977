"""The paged-serving operators, case by case: their plain forms in elementary torch operations, the calls
of the library that compute the same, and their results from the definition in 64 bits.

kind "plan"   block tables, slot maps and positions of a step from the requests' lengths
kind "rope"   rotary positions with one or several axes on q and k, and its inverse (its gradient)
kind "chunk"  new K/V rows into 4-bit pages through a slot map, then the requests' pages as fp16 planes
kind "attn"   attention of ragged queries over 4-bit pages

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
        # a decode step of 256 requests: one row each, the call that a server makes every step
        {"name": "plan_decode", "kind": "plan", "reqs": 256, "fresh": 1, "page_rows": 16, "max_pages": 2048,
         "finished": 0},
        # a step that mixes decodes, prompt chunks and finished requests
        {"name": "plan_mixed", "kind": "plan", "reqs": 4096, "fresh": 250, "page_rows": 32, "max_pages": 256,
         "finished": 7},
        # q and k of one decode step of 32 slots, one axis, fp32 activations
        {"name": "rope_decode", "kind": "rope", "dtype": "f32", "tokens": 32, "hq": 16, "hkv": 2, "hd": 256,
         "rd": 256, "axes": 1, "interleaved": False, "adjacent": False, "inverse": False},
        # a prompt of 8192 tokens with images and video: three axes, a quarter of each head rotated
        {"name": "rope_video", "kind": "rope", "dtype": "bf16", "tokens": 8192, "hq": 16, "hkv": 2, "hd": 256,
         "rd": 64, "axes": 3, "interleaved": True, "adjacent": False, "inverse": False},
        # the gradient of q and k of a long batch of text
        {"name": "rope_grad", "kind": "rope", "dtype": "f16", "tokens": 20011, "hq": 32, "hkv": 8, "hd": 128,
         "rd": 128, "axes": 1, "interleaved": False, "adjacent": True, "inverse": True},
        # speculative decoding's few rows over short caches
        {"name": "chunk_rows", "kind": "chunk", "dtype": "f32", "reqs": 8, "cached": 61, "fresh": 3, "hkv": 2,
         "hd": 64, "page_rows": 16},
        # the next 2048 rows of a prompt whose first 6144 are cached
        {"name": "chunk_prompt", "kind": "chunk", "dtype": "f32", "reqs": 1, "cached": 6144, "fresh": 2048,
         "hkv": 2, "hd": 256, "page_rows": 64},
        # chunks of several prompts at once
        {"name": "chunk_batch", "kind": "chunk", "dtype": "bf16", "reqs": 12, "cached": 9000, "fresh": 517,
         "hkv": 8, "hd": 128, "page_rows": 32},
        # one short request: latency alone
        {"name": "attn_one", "kind": "attn", "dtype": "f16", "reqs": 1, "rows": 600, "ragged": False, "nq": 1,
         "hq": 8, "hkv": 2, "hd": 64, "page_rows": 16, "sink": 0, "win": 0},
        # 32 slots of 32768 keys, the decode that the benchmark times over planes
        {"name": "attn_32x32768", "kind": "attn", "dtype": "bf16", "reqs": 32, "rows": 32768, "ragged": False,
         "nq": 1, "hq": 16, "hkv": 2, "hd": 256, "page_rows": 64, "sink": 0, "win": 0},
        # requests of every length, some rows to verify a draft, fp32 activations
        {"name": "attn_ragged", "kind": "attn", "dtype": "f32", "reqs": 199, "rows": 9001, "ragged": True, "nq": 4,
         "hq": 32, "hkv": 8, "hd": 128, "page_rows": 16, "sink": 0, "win": 0},
        # sinks and a recent window over long requests
        {"name": "attn_window", "kind": "attn", "dtype": "bf16", "reqs": 128, "rows": 16000, "ragged": True,
         "nq": 1, "hq": 16, "hkv": 2, "hd": 256, "page_rows": 32, "sink": 4, "win": 1024},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["plan", "rope", "chunk", "attn", "attn"])
    page_rows = rng.choice([16, 32, 64, 128, 256])
    if kind == "plan":
        reqs = _log(rng, 1, 4096)
        return {"kind": kind, "reqs": reqs, "fresh": _log(rng, 1, min(4096, 1000000 // reqs)),
                "page_rows": page_rows, "max_pages": _log(rng, 512, 2048) if reqs <= 512 else 256,
                "finished": rng.choice([0, 3, 5])}
    dtype = rng.choice(["f32", "f16", "bf16"])
    hd = rng.choice([64, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 8, 16])
    if kind == "rope":
        axes = rng.choice([1, 1, 2, 3, 4])
        return {"kind": kind, "dtype": dtype, "tokens": _log(rng, 1, max(1, 80000000 // (hd * (hq + hkv) * BYTES[dtype] // 2))),
                "hq": hq, "hkv": hkv, "hd": hd, "rd": rng.choice([hd, hd // 2, 64]), "axes": axes,
                "interleaved": axes > 1 and rng.random() < 0.5, "adjacent": rng.random() < 0.5,
                "inverse": rng.random() < 0.4}
    if kind == "chunk":
        most = 6 * 1024 * 1024 * 16 // (hkv * hd)  # rows, so that no case costs more than the largest listed one
        reqs = _log(rng, 1, 64)
        rows = _log(rng, 2, max(2, min(32768, most // reqs // 4)))
        fresh = _log(rng, 1, rows)
        return {"kind": kind, "dtype": dtype, "reqs": reqs, "cached": rows - fresh, "fresh": fresh, "hkv": hkv, "hd": hd,
                "page_rows": page_rows}
    rows = _log(rng, 1, 32768)
    most = 32 * 32768 * 512 // (hkv * hd * rows)
    nq = rng.choice([1, 1, 1, 2, 5])
    reqs = _log(rng, 1, max(1, min(256, most // (2 * max(1, hq // hkv * nq // 8)))))
    sink, win = rng.choice([(0, 0), (0, 0), (4, 1024), (0, 333), (37, 61)])
    return {"kind": kind, "dtype": dtype, "reqs": reqs, "rows": rows, "ragged": rng.random() < 0.7, "nq": nq, "hq": hq,
            "hkv": hkv, "hd": hd, "page_rows": page_rows, "sink": sink, "win": win}


# ------------------------------------------------- lengths that a case stands for

def _spread(n, top, floor=0):
    """n lengths up to `top`, even in their logarithm, from one row up; every seventh of many is `floor`."""
    i = np.arange(n)
    v = np.maximum(1, np.rint(np.exp(np.log(max(top, 1)) * (i + 1) / n))).astype(np.int64)
    return np.where((i % 7 == 3) & (n >= 8), floor, v)


def _plan_lengths(c):
    i = np.arange(c["reqs"])
    most = c["max_pages"] * c["page_rows"]
    # a step of decodes; a step with prompt chunks has one for each third request
    fresh = np.ones(c["reqs"], np.int64) if c["fresh"] == 1 else np.where(i % 3 == 0, 1 + (i * 7919) % c["fresh"], 1)
    fresh = np.minimum(fresh, most)
    cached = (i * 104729 + 11) % np.maximum(1, most - fresh)
    if c["finished"]:
        fresh = np.where(i % c["finished"] == 2, -1, fresh)
    return cached, fresh


def _attn_lengths(c):
    if not c["ragged"]:
        rows = np.full(c["reqs"], c["rows"])
        return rows, np.minimum(c["nq"], rows)
    rows = _spread(c["reqs"], c["rows"])
    return rows, np.minimum(1 + np.arange(c["reqs"]) % c["nq"], np.maximum(rows, 1))


def _chunk_lengths(c):
    i = np.arange(c["reqs"])
    return np.maximum(0, c["cached"] - 5 * i), np.maximum(1, c["fresh"] - 3 * i)


def _visible(rows, nq, sink, win):
    """Rows of a request that any of its queries attends."""
    if win <= 0:
        return rows
    lo = np.maximum(0, rows - nq - win + 1)
    return np.where(rows > 0, np.minimum(lo, sink) + rows - lo, 0)


def work(case):
    c = case
    if c["kind"] == "plan":
        cached, fresh = _plan_lengths(c)
        P, grow = c["page_rows"], np.maximum(fresh, 0)
        popped = -(-(cached + grow) // P) - -(-cached // P)
        pushed = np.where(fresh < 0, -(-cached // P), 0)
        return {"bytes": int(16 * c["reqs"] + 8 * grow.sum() + 8 * popped.sum() + 8 * pushed.sum()), "flops": 0}
    size = BYTES[c["dtype"]]
    if c["kind"] == "rope":
        n = c["tokens"] * (c["hq"] + c["hkv"])
        return {"bytes": 2 * n * c["hd"] * size + 4 * c["axes"] * c["tokens"], "flops": 3 * n * c["rd"]}
    if c["kind"] == "chunk":
        cached, fresh = _chunk_lengths(c)
        row = c["hkv"] * (18 * c["hd"] + 64) // 16
        new, rows = int(fresh.sum()), int((cached + fresh).sum())
        return {"bytes": new * c["hkv"] * c["hd"] * 2 * size + (new + rows) * row + rows * c["hkv"] * c["hd"] * 4,
                "flops": 0}
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


def prepare(case, seed):
    c = case
    rng = np.random.default_rng(seed)
    g = torch.Generator("cuda").manual_seed(seed)
    s = dict(c)
    if c["kind"] == "plan":
        cached, fresh = _plan_lengths(c)
        mix = rng.permutation(c["reqs"])
        cached, fresh = cached[mix], fresh[mix]
        P, R = c["page_rows"], c["reqs"]
        used = -(-cached // P)
        need = -(-(cached + np.maximum(fresh, 0)) // P) - used
        n_pages = int(used.sum() + need.sum() + R)
        order, table = rng.permutation(n_pages), np.full((R, c["max_pages"]), -1, np.int64)
        table[np.arange(c["max_pages"]) < used[:, None]] = order[:used.sum()]
        ring, head = np.full(n_pages, -1, np.int64), int(rng.integers(n_pages))
        free = n_pages - int(used.sum())
        ring[(head + np.arange(free)) % n_pages] = order[used.sum():]
        T = int(np.maximum(fresh, 0).sum()) + 5  # the batch is padded: 5 tokens of no request
        s.update(cached=_int(cached), fresh=_int(fresh), ring=_int(ring), state=_int([head, free]), table=_int(table),
                 T=T, state_out=torch.zeros(3, dtype=torch.int32, device="cuda"),
                 lens=torch.zeros(R, dtype=torch.int32, device="cuda"),
                 cu=torch.zeros(R + 1, dtype=torch.int32, device="cuda"),
                 slots=torch.zeros(T, dtype=torch.int32, device="cuda"),
                 pos=torch.zeros(T, dtype=torch.int32, device="cuda"))
        return s
    dt = DTYPES[c["dtype"]]
    rand = lambda *shape: torch.randn(shape, device="cuda", generator=g).to(dt)  # noqa: E731
    if c["kind"] == "rope":
        T, A, half = c["tokens"], c["axes"], c["rd"] // 2
        qkv = rand(T, c["hq"] + 2 * c["hkv"], c["hd"])  # one projection's output; v is left alone
        pos = rng.integers(0, 4096, (A, T))
        pos[0] = rng.integers(0, 1 << 17) + np.arange(T)
        sections = [half - (A - 1) * (half // (A + 1)), *[half // (A + 1)] * (A - 1)]
        inv_freq = 1e6 ** (-np.arange(half) / half)
        i, edge = np.arange(half), np.cumsum(sections)
        axis = i % A
        axis = np.where(i < A * np.array(sections)[axis], axis, 0) if c["interleaved"] else np.searchsorted(edge, i, "right")
        s.update(q=qkv[:, :c["hq"]], k=qkv[:, c["hq"]:c["hq"] + c["hkv"]], pos=_int(pos),
                 inv_freq=torch.tensor(inv_freq, dtype=torch.float64, device="cuda"), axis=torch.as_tensor(axis, device="cuda"),
                 q_out=torch.empty(T, c["hq"], c["hd"], dtype=dt, device="cuda"),
                 k_out=torch.empty(T, c["hkv"], c["hd"], dtype=dt, device="cuda"),
                 # what fa.rope_table makes once for a model: each pair's turns per position and its axis
                 table=_turns(inv_freq, axis))
        return s
    if c["kind"] == "chunk":
        cached, fresh = _chunk_lengths(c)
        rows = cached + fresh
        table, n = _table(rng, rows, c["page_rows"])
        T = int(fresh.sum())
        req = np.repeat(np.arange(c["reqs"]), fresh)
        at = np.arange(T) - np.repeat(np.cumsum(fresh) - fresh, fresh) + cached[req]
        slots = table[req, at // c["page_rows"]] * c["page_rows"] + at % c["page_rows"]
        max_seq = int(rows.max()) + 3
        plane = (c["hkv"] * max_seq * c["hd"] * 2 + 255) // 256 * 256
        s.update(pages=_pool(g, n, c["hkv"], c["page_rows"], c["hd"]), table=_int(table), lens=_int(rows), slots=_int(slots),
                 req=torch.as_tensor(req, device="cuda"), at=torch.as_tensor(at, device="cuda"),
                 k=rand(T, c["hkv"], c["hd"]), v=rand(T, c["hkv"], c["hd"]), max_seq=max_seq,
                 k_planes=torch.zeros(c["reqs"] * plane, dtype=torch.uint8, device="cuda"),
                 v_planes=torch.zeros(c["reqs"] * plane, dtype=torch.uint8, device="cuda"))
        return s
    rows, nq = _attn_lengths(c)
    mix = rng.permutation(c["reqs"])
    rows, nq = rows[mix], nq[mix]
    table, n = _table(rng, rows, c["page_rows"])
    T = int(nq.sum())
    s.update(pages=_pool(g, n, c["hkv"], c["page_rows"], c["hd"]), table=_int(table), lens=_int(rows),
             cu=_int(np.concatenate([[0], np.cumsum(nq)])), q=rand(T, c["hq"], c["hd"]), n_q=int(nq.max()),
             req=torch.as_tensor(np.repeat(np.arange(c["reqs"]), nq), device="cuda"),
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
    return {"plan": _run_plan, "rope": _run_rope, "chunk": _run_chunk, "attn": _run_attn}[s["kind"]](s)


def _run_plan(s):
    P = s["page_rows"]
    if own:
        import causal_gqa_flash_attn_gb300 as fa
        fa.page_plan(s["cached"], s["fresh"], s["ring"], s["state"], s["table"], s["state_out"], s["lens"], s["cu"],
                     s["slots"], s["pos"], page_rows=P)
        return {k: s[k] for k in ("ring", "state_out", "table", "lens", "cu", "slots", "pos")}
    cached, fresh, n = s["cached"].long(), s["fresh"].long(), s["ring"].numel()
    head, free = s["state"].long()
    grow = fresh.clamp(min=0)
    used = (cached + P - 1) // P
    need = (cached + grow + P - 1) // P - used
    upto = need.cumsum(0)
    fits = (need == 0) | (upto <= free)
    taken = torch.where(fits, need, 0)
    ring, table = s["ring"].clone(), s["table"].clone()
    # pages of finished requests go behind the ring's last
    back = torch.where(fresh < 0, used, 0)
    col = torch.arange(table.shape[1], device="cuda")
    give = (col < back.unsqueeze(1)).nonzero(as_tuple=True)
    place = (back.cumsum(0) - back)[give[0]] + give[1]
    ring[(head + free + place) % n] = table[give]
    # each request's new pages, in request order
    new = col.sub(used.unsqueeze(1))
    take = ((new >= 0) & (new < taken.unsqueeze(1))).nonzero(as_tuple=True)
    place = (upto - need)[take[0]] + new[take]
    table[take] = s["ring"][(head + place) % n]
    lens = torch.where(fresh < 0, 0, torch.where(fits, cached + grow, cached))
    cu = torch.cat([grow.new_zeros(1), grow.cumsum(0)])
    token = torch.arange(s["T"], device="cuda")
    req = torch.searchsorted(cu[1:], token, right=True)
    live = req < fresh.numel()
    req = req.clamp(max=fresh.numel() - 1)
    pos = cached[req] + token - cu[req]
    page = table[req, (pos // P).clamp(max=table.shape[1] - 1)].long()
    slots = torch.where(live & fits[req], page * P + pos % P, -1)
    state = torch.stack([(head + taken.sum()) % n, free - taken.sum() + back.sum(), need.sum() - taken.sum()])
    return {"ring": ring, "state_out": state.int(), "table": table, "lens": lens.int(), "cu": cu.int(), "slots": slots.int(),
            "pos": torch.where(live, pos, 0).int()}


def _run_rope(s):
    if own:
        import causal_gqa_flash_attn_gb300 as fa
        fa.rope(s["q"], s["k"], s["q_out"], s["k_out"], s["pos"], s["table"], adjacent=s["adjacent"], inverse=s["inverse"])
        return {"q": s["q_out"], "k": s["k_out"]}
    angle = s["pos"].double()[s["axis"]].T * s["inv_freq"]  # [tokens][pairs]; 64 bits: far positions
    if s["inverse"]:
        angle = -angle
    cos, sin, rd = angle.cos().float().unsqueeze(1), angle.sin().float().unsqueeze(1), s["rd"]

    def turn(x):
        y = x.float()
        r = y[..., :rd].unflatten(-1, (-1, 2)).transpose(-1, -2) if s["adjacent"] else y[..., :rd].unflatten(-1, (2, -1))
        a, b = r[..., 0, :], r[..., 1, :]
        r = torch.stack([a * cos - b * sin, a * sin + b * cos], -2)
        r = (r.transpose(-1, -2) if s["adjacent"] else r).flatten(-2)
        return torch.cat([r, y[..., rd:]], -1).to(x.dtype)

    return {"q": turn(s["q"]), "k": turn(s["k"])}


def _planes(s):
    """The fp16 planes [requests][hkv][max_seq][hd] as the values they hold."""
    n, rows = s["reqs"], s["hkv"] * s["max_seq"] * s["hd"]
    cut = lambda p: p.view(n, -1)[:, :2 * rows].view(torch.float16).view(n, s["hkv"], s["max_seq"], s["hd"])  # noqa: E731
    return {"k": cut(s["k_planes"]), "v": cut(s["v_planes"])}


def _run_chunk(s):
    if own:
        import causal_gqa_flash_attn_gb300 as fa
        fa.paged_append(s["k"], s["v"], s["slots"], s["pages"], page_rows=s["page_rows"])
        fa.paged_gather(s["pages"], s["table"], s["lens"], s["k_planes"], s["v_planes"], n_kv_heads=s["hkv"],
                        head_dim=s["hd"], page_rows=s["page_rows"], max_seq=s["max_seq"])
        return _planes(s)
    k, v = _rows_of(s)
    live = (torch.arange(s["max_seq"], device="cuda") < s["lens"].unsqueeze(1))[:, None, :, None]
    made = {}
    for name, old, new in (("k", k, s["k"]), ("v", v, s["v"])):
        codes, scales, factors = _quantise(new.float())
        x = (codes.float() - 8).unflatten(-1, (-1, 32)) * (scales.float() * factors.unsqueeze(-1)).unsqueeze(-1)
        plane = torch.zeros(live.shape[0], s["hkv"], s["max_seq"], s["hd"], device="cuda")
        n = min(s["max_seq"], old.shape[2])
        plane[:, :, :n] = old[:, :, :n]
        plane[s["req"], :, s["at"]] = x.flatten(-2)
        made[name] = torch.where(live, plane, 0.0).half()
    return made


def _rows_of(s):
    """K and V of the requests' pages [requests][hkv][rows][hd] fp32; rows of no page are some page's."""
    P, hd = s["page_rows"], s["hd"]
    atoms = s["pages"].view(-1, s["hkv"], P // 16, 18 * hd + 64)
    atoms = atoms[s["table"].long().clamp(min=0)].transpose(1, 2)  # [requests][hkv][pages][groups][bytes]
    k, v = atoms.split(9 * hd + 32, -1)
    return _unpack_part(k, hd, False).flatten(2, 4), _unpack_part(v, hd, True).flatten(2, 4)


def _run_attn(s):
    if own:
        import causal_gqa_flash_attn_gb300 as fa
        fa.paged_attn(s["q"], s["out"], s["cu"], s["lens"], s["table"], s["pages"], n_kv_heads=s["hkv"],
                      page_rows=s["page_rows"], sink=s["sink"], win=s["win"], lse=s["lse"], workspace=s["workspace"])
        return {"out": s["out"], "lse": s["lse"]}
    k, v = _rows_of(s)
    R, hkv, rows, hd = k.shape
    cu, lens = s["cu"].long(), s["lens"].long()
    nth = torch.arange(s["req"].numel(), device="cuda") - cu[s["req"]]  # a token's place in its request
    q = torch.zeros(R, s["n_q"], s["hq"], hd, device="cuda")
    q[s["req"], nth] = s["q"].float()
    q = q.view(R, s["n_q"], hkv, -1, hd).permute(0, 2, 1, 3, 4)  # [requests][hkv][queries][group][hd]
    score = (q.flatten(2, 3) @ k.transpose(-1, -2)) / math.sqrt(hd)
    score = score.view(R, hkv, s["n_q"], -1, rows)
    j = torch.arange(rows, device="cuda")
    p = (lens - (cu[1:] - cu[:-1])).unsqueeze(1) + torch.arange(s["n_q"], device="cuda")
    p = p[:, None, :, None, None]
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


def exact(case, seed):
    c = case
    if c["kind"] == "plan":
        return None  # whole numbers
    s = prepare(c, seed)
    if c["kind"] == "rope":
        made = {}
        rd, A = c["rd"], s["axis"].tolist()
        angle = torch.stack([s["pos"][a].double() * f for a, f in zip(A, s["inv_freq"].tolist())], 1)
        z = torch.polar(torch.ones_like(angle), -angle if c["inverse"] else angle).unsqueeze(1)
        for name in ("q", "k"):
            x = s[name].double().clone()
            i = torch.arange(rd // 2, device="cuda")
            re, im = (2 * i, 2 * i + 1) if c["adjacent"] else (i, i + rd // 2)
            y = torch.complex(x[..., re], x[..., im]) * z
            x[..., re], x[..., im] = y.real, y.imag
            made[name] = x
        return made
    if c["kind"] == "chunk":
        cached, fresh = _chunk_lengths(c)
        made = {n: torch.zeros(c["reqs"], c["hkv"], s["max_seq"], c["hd"], dtype=torch.float64, device="cuda") for n in "kv"}
        t = 0
        for r in range(c["reqs"]):
            if cached[r]:
                made["k"][r, :, :cached[r]], made["v"][r, :, :cached[r]] = _request(s, r, 0, int(cached[r]))
            for n in "kv":
                x = s[n][t:t + fresh[r]].float().cpu().numpy().reshape(int(fresh[r]), c["hkv"], -1, 32)
                d = (np.abs(x).max(-1) / np.float32(-8)).astype(np.float32)
                inv = np.divide(np.float32(1), d, out=np.zeros_like(d), where=d != 0)
                code = np.clip(np.rint(x * inv[..., None]) + 8, 0, 15)
                top = np.abs(d).max(-1).astype(np.float64)
                e = np.floor(np.log2(np.where(top > 0, top, 1.0)))
                scale = (d.astype(np.float64) * 2.0 ** -e[..., None]).astype(np.float16).astype(np.float64) * 2.0 ** e[..., None]
                rows = torch.as_tensor((code - 8) * scale[..., None]).flatten(-2).transpose(0, 1)
                made[n][r, :, cached[r]:cached[r] + fresh[r]] = rows.cuda()
            t += int(fresh[r])
        return made
    lens, cu = s["lens"].tolist(), s["cu"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full((c["hq"], s["q"].shape[0]), -math.inf, dtype=torch.float64, device="cuda")
    for r in range(c["reqs"]):
        if not lens[r]:
            continue
        k, v = _request(s, r, 0, lens[r])
        k, v = (x.repeat_interleave(c["hq"] // c["hkv"], 0) for x in (k, v))
        for t in range(cu[r], cu[r + 1]):
            p = lens[r] - cu[r + 1] + t
            keep = torch.arange(p + 1, device="cuda")
            if c["win"] > 0:
                keep = keep[(keep < c["sink"]) | (keep > p - c["win"])]
            x = torch.einsum("hd,hjd->hj", s["q"][t].double(), k[:, keep]) / math.sqrt(c["hd"])
            lse[:, t] = torch.logsumexp(x, -1)
            out[t] = torch.einsum("hj,hjd->hd", torch.exp(x - lse[:, t:t + 1]), v[:, keep])
    return {"out": out, "lse": lse}
