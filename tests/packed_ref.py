"""Packed attention and its gradient from the definition in 64 bits, document by document and head by head:
the reference of the packed tests, with bounds of what rounding may do to each result. It shares no code
with the library."""
from __future__ import annotations

import math

import torch

EPS = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}  # half a step, relative
# Half a step of the smallest numbers: below 2^-14 binary16's lie 2^-24 apart, below 2^-126 bfloat16's 2^-133.
LEAST = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def seen(n, prefix=0, sink=0, win=0):
    """[query][key] of a document of n tokens."""
    i, j = torch.arange(n)[:, None], torch.arange(n)[None, :]
    see = j <= i
    if win > 0:
        see = see & ((j < sink) | (j > i - win))
    return see | (j < prefix)


def document(q, k, v, slope, *, prefix=0, sink=0, win=0, scale=0.0, cap=0.0, dout=None):
    """One head of one document: q, k, v [n][hd] in 64 bits. A dict of out, lse (and dq, dk, dv), each with
    a bound of the error that the library's roundings may make: of the weights and of the scores' gradients
    to the inputs' type (eps), of sums and scores in 32 bits; the rounding of the result itself is not in it."""
    n, hd = q.shape
    scale = scale or 1 / math.sqrt(hd)
    see = seen(n, prefix, sink, win).to(q.device)
    s = q @ k.T * scale
    size = q.abs() @ k.abs().T * scale  # what a score's sum adds up
    x, down = s, torch.ones_like(s)
    if cap > 0:
        x = cap * torch.tanh(s / cap)
        down = 1 - torch.tanh(s / cap) ** 2
    far = (torch.arange(n)[:, None] - torch.arange(n)[None, :]).abs().to(q)
    x = x - slope * far
    x = torch.where(see, x, -math.inf)
    lse = torch.logsumexp(x, -1)
    w = torch.exp(x - lse[:, None])
    # a score: its sum of hd products in 32 bits (the tensor cores cut), the cap's and the bias's arithmetic
    ds = 2.0 ** -21 * (size + cap + slope * far + lse.abs()[:, None] + 1)
    ds = torch.where(see, ds, 0.0)
    wrong = w * ds
    made = {"out": w @ v, "lse": lse, "out_err": 2 * wrong @ v.abs(), "lse_err": wrong.sum(-1),
            "out_sum": w @ v.abs()}
    if dout is not None:
        out = made["out"]
        dw = dout @ v.T
        D = (dout * out).sum(-1, keepdim=True)
        t = w * (dw - D) * down
        # D from the rounded out, and sums in 32 bits
        D_sum = (dout * out).abs().sum(-1, keepdim=True)
        rest = 2.0 ** -21 * (dout.abs() @ v.abs().T + D_sum)
        # (down: 1 - tanh^2 is off by 2^-52 in 64 bits, and the library's is 2^-61 at least)
        made.update(dq=scale * t @ k, dk=scale * t.T @ q, dv=w.T @ dout,
                    t=t, w=w, D_sum=D_sum, t_err=2 * t.abs() * ds + w * rest * (down + 2.0 ** -50) + w * (dw - D).abs() * 2.0 ** -20,
                    w_err=2 * wrong, scale=scale, down=down)
    return made


def packed(q, k, v, cu, slopes=None, prefix=None, dout=None, **rule):
    """q [T][Hq][hd], k, v [T][Hkv][hd] of fp16 or bf16: dict of out, lse (dq, dk, dv) and of their bounds
    (name + "_err") in 64 bits, zeros for padding."""
    eps, least, narrow = EPS[q.dtype], LEAST[q.dtype], q.dtype == torch.float16
    T, hq, hd = q.shape
    g = hq // k.shape[1]
    wide = {n: t.double() for n, t in (("q", q), ("k", k), ("v", v))}
    names = ("out", "dq", "dk", "dv") if dout is not None else ("out",)
    made = {}
    for n in names:
        like = q if n in ("out", "dq") else k
        made[n] = torch.zeros(like.shape, dtype=torch.float64, device=q.device)
        made[n + "_err"] = torch.zeros_like(made[n])
    made["lse"] = torch.zeros(hq, T, dtype=torch.float64, device=q.device)
    made["lse_err"] = torch.zeros_like(made["lse"])
    for d in range(len(cu) - 1):
        at = slice(cu[d], cu[d + 1])
        if cu[d + 1] <= cu[d]:
            continue
        for h in range(hq):
            do = dout[at, h].double() if dout is not None else None
            slope = float(slopes[h]) if slopes is not None else 0.0
            p = min(int(prefix[d]), cu[d + 1] - cu[d]) if prefix is not None else 0
            qd, kd, vd = wide["q"][at, h], wide["k"][at, h // g], wide["v"][at, h // g]
            r = document(qd, kd, vd, slope, prefix=p, dout=do, **rule)
            made["out"][at, h], made["lse"][h, at] = r["out"], r["lse"]
            # weights rounded to the type (fp16: to its smallest numbers at worst), then the result
            made["out_err"][at, h] = (r["out_err"] + (eps + 2.0 ** -19) * r["out_sum"]
                                      + least * (kd.shape[0] ** 0.5) * vd.abs().amax(0)
                                      + eps * r["out"].abs() + least)
            made["lse_err"][h, at] = r["lse_err"] + 2.0 ** -22 * (r["lse"].abs() + 1)
            if do is None:
                continue
            # t: from w and D, where D = dout . out has out's rounding, then rounded to the type
            D_err = (do.abs() * made["out_err"][at, h]).sum(-1, keepdim=True)
            t_err = r["t_err"] + r["w"] * D_err * r["down"] + eps * r["t"].abs()
            # (fp16: t is scaled so that what it can lose at its small end is 2^-38 of |dout| |v|)
            if narrow:
                t_err = t_err + 2.0 ** -37 * do.norm(dim=-1).max() * vd.norm(dim=-1).max()
            w_err = r["w_err"] + eps * r["w"] + (2.0 ** -39 if narrow else 2.0 ** -126)
            s = r["scale"]
            made["dq"][at, h] = r["dq"]
            made["dq_err"][at, h] = s * t_err @ kd.abs() + 2.0 ** -19 * s * r["t"].abs() @ kd.abs()
            made["dk"][at, h // g] += r["dk"]
            made["dk_err"][at, h // g] += s * t_err.T @ qd.abs() + 2.0 ** -19 * s * r["t"].abs().T @ qd.abs()
            made["dv"][at, h // g] += r["dv"]
            made["dv_err"][at, h // g] += w_err.T @ do.abs() + 2.0 ** -19 * r["w"].T @ do.abs()
    for n in names[1:]:
        made[n + "_err"] += eps * made[n].abs() + least
    return made
