"""Paged attention with capped scores and a bias by distance, and the append that rotates on the way, on the GPU:
against the definition in 64 bits, against the calls that they stand for, and together with the packed calls."""
import math

import numpy as np
import pytest
import torch

import packed_ref
import paged_ref as ref
from gpu_util import check_guards, fa, guarded

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def ints(a):
    return torch.tensor(np.asarray(a, np.int32), dtype=torch.int32, device="cuda")


# ----------------------------------------------------------- scored attention

def pages_of(rng, rows, hkv, hd, page_rows, strong=1.0):
    """Pages with random rows for requests of these lengths, the values that they hold [hkv][rows][hd] in 64
    bits, and their table."""
    need = [-(-n // page_rows) for n in rows]
    total = sum(need) + 2
    order = rng.permutation(total)
    table = np.full((len(rows), max(max(need), 1)), -1)
    pages = fa().alloc_pages(total, hkv, hd, page_rows)
    pages.fill_(0x7f)  # rows that nobody wrote: scales of NaN
    held, at = [], 0
    for r, n in enumerate(rows):
        table[r, :need[r]] = order[at:at + need[r]]
        at += need[r]
        x = [(rng.standard_normal((n, hkv, hd)) * strong).astype(np.float32) for _ in range(2)]
        if n:
            slots = table[r, np.arange(n) // page_rows] * page_rows + np.arange(n) % page_rows
            fa().paged_append(torch.from_numpy(x[0]).cuda(), torch.from_numpy(x[1]).cuda(), ints(slots), pages,
                              page_rows=page_rows)
        held.append([ref.decode(*ref.encode(y)) for y in x])
    return pages, table, held


def attend(q, first, k, v, cap, slopes, sink, win, scale):
    """Queries q [n][Hq][hd] at positions first.. over rows k, v [L][Hkv][hd]: out, lse, the sums of w |v|,
    what the scores' 32-bit sums add up, and what K's codes add to that with their offset."""
    n, hq, hd = q.shape
    g = hq // k.shape[1]
    out, lse, size, off = np.zeros(q.shape), np.full((hq, n), -math.inf), np.zeros(q.shape), np.zeros((hq, n))
    codes = np.zeros((hq, n))
    step = np.repeat(np.abs(k).reshape(*k.shape[:2], hd // 32, 32).max(-1) / 7, 32, -1)
    for i in range(n):
        p, j = first + i, np.arange(k.shape[0])
        see = j <= p
        if win > 0:
            see &= (j < sink) | (j > p - win)
        if not see.any():
            continue
        for h in range(hq):
            kk, vv = k[see, h // g], v[see, h // g]
            s = kk @ q[i, h] * scale
            x = cap * np.tanh(s / cap) if cap else s
            x = x - (slopes[h] * (p - j[see]) if slopes is not None else 0.0)
            lse[h, i] = x.max() + np.log(np.exp(x - x.max()).sum())
            w = np.exp(x - lse[h, i])
            out[i, h], size[i, h] = w @ vv, w @ np.abs(vv)
            # sums of hd products, the bias's and the reference's arithmetic (in 2^-24 steps, cut by the
            # tensor cores): relative to what is added up
            e = np.abs(kk) @ np.abs(q[i, h]) * scale + np.abs(x) + (slopes[h] * (p - j[see]) if slopes is not None else 0)
            off[h, i] = (w * e).sum() + abs(lse[h, i]) + 1
            codes[h, i] = (w * (16 * step[see, h // g] @ np.abs(q[i, h]) * scale)).sum()
    return out, lse, size, off, codes


def run_paged(rng, dtype, rows, nq, hq, hkv, hd, page_rows, cap=0.0, bias=False, sink=0, win=0, gain=1.0, scale=0.0):
    m = fa()
    pages, table, held = pages_of(rng, rows, hkv, hd, page_rows)
    cu = np.concatenate([[0], np.cumsum(nq)])
    T = int(cu[-1]) + 2
    q = ref.round_type(rng.standard_normal((T, hq, hd)) * gain, dtype)
    slopes = np.float32(0.5) ** np.arange(1, hq + 1, dtype=np.float32) if bias else None
    out = guarded((T, hq, hd), DT[dtype], fill=-7.0)
    lse = guarded((hq, T), torch.float32, fill=-7.0)
    ws = guarded(m.paged_attn_workspace_bytes(hd), torch.uint8)
    m.paged_attn(torch.from_numpy(q).to(DT[dtype]).cuda(), out, ints(cu), ints(rows), ints(table), pages, n_kv_heads=hkv,
                 page_rows=page_rows, sink=sink, win=win, scale=scale, cap=cap, lse=lse, workspace=ws,
                 slopes=None if slopes is None else torch.from_numpy(slopes).cuda())
    torch.cuda.synchronize()
    check_guards(("out", out), ("lse", lse), ("workspace", ws))
    assert m.get_device_error() == m.OK
    got, glse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert (got[cu[-1]:] == -7.0).all() and (glse[:, cu[-1]:] == -7.0).all()
    half = ref.HALF_STEP[dtype]
    for r, n in enumerate(rows):
        a, b = cu[r], cu[r + 1]
        want, wlse, size, off, codes = attend(q[a:b], n - (b - a), *held[r], cap, slopes, sink, win,
                                       scale or 1 / math.sqrt(hd))
        # scores: 2^-21 of what they add up; the tanh 2^-21 of the cap (2^-23 for fp32, by tanhf)
        ds = off * 2.0 ** -21 + cap * (2.0 ** -23 if dtype == "f32" else 2.0 ** -21)
        weights = {"f32": 2.0 ** -20, "f16": 2.0 ** -20, "bf16": 2.0 ** -10}[dtype]  # two roundings to binary16 in bf16
        tol = size * (weights * (1 + 2.0 ** -11) + 2 * ds.T[:, :, None]) + 2.0 ** -24
        # V's codes enter with their offset 8, which is taken out of the sum: its terms are up to 16 code steps
        # (a seventh of a block's largest value or less) times the weights, 1 in all, and each addition of 16 rows,
        # of the pieces and of the joins may lose a step of 2^-23 of it
        step = np.abs(held[r][1]).reshape(n, hkv, hd // 32, 32).max(-1) / 7 if n else np.zeros((1, hkv, hd // 32))
        step = np.repeat(np.repeat(step, 32, -1), hq // hkv, 1).max(0)
        tol = tol + 2 * (-(-n // 16) + 40) * 2.0 ** -23 * 16 * step
        # what is rounded at the end is the computed value, up to |want| + tol (a request of one row has all
        # of its weights off alike, so that both errors do add up)
        tol = tol + half * (np.abs(want) + tol)
        assert (np.abs(got[a:b] - want) <= tol).all(), (r, np.abs(got[a:b] - want).max())
        live = np.isfinite(wlse)
        assert np.array_equal(live, np.isfinite(glse[:, a:b])) and (glse[:, a:b][~live] == -math.inf).all()
        # K's codes enter the products with 16-bit queries with their offset 8, too: terms of up to 16 code steps
        # (a seventh of a block's largest value or less), whose sum is cut like the scores' own
        ds = ds + (0.0 if dtype == "f32" else codes * 2.0 ** -21)
        assert (np.abs(glse[:, a:b][live] - wlse[live]) <= ds[live] + 2.0 ** -21).all(), r


@pytest.mark.parametrize("cap,bias", [(0.0, True), (20.0, False), (3.0, True)])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_scored(dtype, hd, cap, bias):
    rng = np.random.default_rng(hd)
    run_paged(rng, dtype, [1, 37, 0, 300, 16, 129], [1, 3, 0, 1, 2, 5], 8, 2, hd, 32, cap, bias, gain=4.0)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,page_rows", [(1, 1, 16), (2, 2, 256), (16, 1, 64), (32, 2, 128)])
def test_groups_and_pages(hq, hkv, page_rows, dtype):
    run_paged(np.random.default_rng(hq), dtype, [90, 555, 2], [1, 2, 1], hq, hkv, 64, page_rows, 10.0, True, gain=3.0)


@pytest.mark.parametrize("sink,win", [(0, 1), (4, 50), (37, 61), (200, 5)])
def test_windows(sink, win):
    for hd in (64, 128, 256):
        run_paged(np.random.default_rng(win), "bf16", [400, 33, 1, 129], [1, 4, 1, 2], 4, 2, hd, 16, 8.0, True, sink, win)


def test_more_queries_than_rows_attend_nothing():
    run_paged(np.random.default_rng(2), "f16", [2, 0], [5, 1], 4, 2, 64, 16, 8.0, True)


def test_many_requests():
    rng = np.random.default_rng(4)
    rows = rng.integers(0, 70, 90)
    run_paged(rng, "bf16", rows, np.minimum(1, rows), 8, 4, 64, 16, 12.0, True)


def test_long_request():
    run_paged(np.random.default_rng(5), "f16", [9000], [1], 4, 1, 128, 64, 30.0, True, gain=5.0)


def test_without_cap_and_slopes_it_is_the_plain_call():
    m = fa()
    rng = np.random.default_rng(6)
    pages, table, _ = pages_of(rng, [500, 60], 2, 128, 32)
    q = torch.randn(2, 8, 128, device="cuda").bfloat16()
    ws = torch.empty(m.paged_attn_workspace_bytes(128), dtype=torch.uint8, device="cuda")
    a, b, c = (torch.empty_like(q) for _ in range(3))
    rest = (ints([0, 1, 2]), ints([500, 60]), ints(table), pages)
    kw = dict(n_kv_heads=2, page_rows=32, workspace=ws)
    m.paged_attn(q, a, *rest, **kw)
    m.paged_attn(q, b, *rest, cap=0.0, slopes=None, **kw)
    # slopes of zeros: the scored kernel, the same scores
    m.paged_attn(q, c, *rest, slopes=torch.zeros(8, device="cuda"), **kw)
    assert torch.equal(a, b)
    # both round their weights: 2^-10 of what they add up each (below 5 here), and the result
    assert ((a.float() - c.float()).abs() <= 2 * 2.0 ** -8 * a.float().abs() + 2 * 2.0 ** -10 * 5).all()


def test_infinite_scores_are_capped():
    """A K row with an infinity (a NaN block) stays a NaN; a very large score is the cap."""
    m = fa()
    pages = m.alloc_pages(1, 1, 64, 16)
    k = torch.zeros(2, 1, 64, device="cuda")
    k[0, 0, 0], k[1, 0, 0] = 2e19, -2e19
    v = torch.ones(2, 1, 64, device="cuda")
    v[1] = -1.0
    m.paged_append(k, v, ints([0, 1]), pages, page_rows=16)
    q = torch.zeros(1, 1, 64, device="cuda")
    q[0, 0, 0] = 1e19
    out, lse = torch.empty_like(q), torch.empty(1, 1, device="cuda")
    m.paged_attn(q, out, ints([0, 1]), ints([2]), ints([[0]]), pages, n_kv_heads=1, page_rows=16, cap=2.0, lse=lse,
                 workspace=torch.empty(m.paged_attn_workspace_bytes(64), dtype=torch.uint8, device="cuda"))
    # scores 2 and -2; v = 1 is stored as 7/8 or 1 by its sign (codes -8 .. 7 of amax / -8)
    a = math.exp(2) / (math.exp(2) + math.exp(-2))
    held = [ref.decode(*ref.encode(x.cpu().numpy()))[0, 0, 0] for x in (v[:1], v[1:])]
    assert abs(lse.item() - math.log(math.exp(2) + math.exp(-2))) < 1e-5
    assert abs(out[0, 0, 0].item() - (a * held[0] + (1 - a) * held[1])) < 1e-5


# ------------------------------------------------------------- rotated append

def rope_case(rng, dtype, T, hq, hkv, hd, rd, axes, spare=0):
    """q, k, v of one projection, positions, a table, slots (some left out) and pages."""
    m = fa()
    wide = torch.randn(T, (hq + 2 * hkv) * hd + spare, device="cuda").to(DT[dtype])
    qkv = wide[:, :(hq + 2 * hkv) * hd].unflatten(1, (-1, hd))
    pos = ints(rng.integers(-5, 1 << 20, (axes, T)))
    sections = [rd // 2 - (axes - 1) * (rd // 2 // (axes + 1))] + [rd // 2 // (axes + 1)] * (axes - 1)
    table = m.rope_table(1e4 ** (-np.arange(rd // 2) / (rd // 2)), sections)
    slots = rng.permutation(4 * 32)[:T]
    slots[rng.random(T) < 0.2] = -1
    pages = m.alloc_pages(4, hkv, hd, 32)
    pages.fill_(0x5a)
    return qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], pos, table, ints(slots), pages


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("hd,rd", [(64, 64), (64, 6), (128, 64), (128, 128), (128, 40), (256, 256), (256, 2), (256, 64)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_rope_append_is_rope_and_append(dtype, hd, rd, adjacent):
    """Bit for bit, for one token and more than a block has."""
    m = fa()
    rng = np.random.default_rng(hd + rd)
    for T, hq, hkv, axes in ((1, 1, 1, 1), (77, 6, 3, min(3, rd // 2)), (33, 16, 2, 1)):
        q, k, v, pos, table, slots, pages = rope_case(rng, dtype, T, hq, hkv, hd, rd, axes, spare=8)
        twin = pages.clone()
        q0, k0 = q.clone(), k.clone()
        qw, kw = torch.empty_like(q0), torch.empty_like(k0)
        m.rope(q, k, qw, kw, pos, table, adjacent=adjacent)
        m.paged_append(kw, v, slots, twin, page_rows=32)
        q_out = guarded(q.shape, q.dtype, fill=-7.0)
        m.rope_append(q, k, v, q_out, pos, table, slots, pages, page_rows=32, adjacent=adjacent)
        torch.cuda.synchronize()
        check_guards(("q_out", q_out))
        assert torch.equal(q_out, qw) and torch.equal(pages, twin)
        assert torch.equal(q, q0) and torch.equal(k, k0)
        # in place, and without q
        twin.fill_(0x5a)
        m.rope_append(None, k, v, None, pos, table, slots, twin, page_rows=32, adjacent=adjacent)
        assert torch.equal(pages, twin)
        m.rope_append(q, k, v, q, pos, table, slots, pages, page_rows=32, adjacent=adjacent)
        assert torch.equal(q, qw) and torch.equal(pages, twin) and torch.equal(k, k0)
    assert m.get_device_error() == m.OK


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("hd,rd", [(64, 64), (128, 40), (128, 6), (256, 256)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_a_pair_turns_with_the_stated_roundings(dtype, hd, rd, adjacent):
    """x0 = fma(u0, c, -(u1 s)) and x1 = fma(u0, s, u1 c) in 32 bits, from the sines and cosines that a pair (1, 0)
    turns into; and the same bits in the pages of the append that rotates."""
    m = fa()
    half, n = rd // 2, 50
    table = m.rope_table(1e4 ** (-np.arange(half) / half))
    pos = ints(np.random.default_rng(rd).integers(-9, 1 << 20, n))
    first = slice(0, rd, 2) if adjacent else slice(0, half)
    second = slice(1, rd, 2) if adjacent else slice(half, rd)
    unit = torch.zeros(n, 1, hd, device="cuda")
    unit[..., first] = 1.0
    m.rope(unit, None, unit, None, pos, table, adjacent=adjacent)
    c, s = unit[..., first], unit[..., second]
    x = torch.randn(n, 3, hd, device="cuda", generator=torch.Generator("cuda").manual_seed(hd + rd)).to(DT[dtype])
    u0, u1 = x[..., first].float(), x[..., second].float()
    # (in 64 bits the product is exact, and the sum is rounded to 53 bits before it is rounded to 24: these values
    # do not lie within 2^-29 of a step from the middle between two)
    fma = lambda a, b, d: (a.double() * b.double() + d.double()).float()  # noqa: E731
    want = x.clone()
    want[..., first] = fma(u0, c, -(u1 * s)).to(DT[dtype])
    want[..., second] = fma(u0, s, u1 * c).to(DT[dtype])
    got = torch.empty_like(x)
    m.rope(x, None, got, None, pos, table, adjacent=adjacent)
    assert torch.equal(got, want)
    slots = ints(np.arange(n))
    pages = [m.alloc_pages(4, 3, hd, 16).fill_(0x5a) for _ in range(2)]
    m.rope_append(None, x, x, None, pos, table, slots, pages[0], page_rows=16, adjacent=adjacent)
    m.paged_append(want, x, slots, pages[1], page_rows=16)
    assert torch.equal(*pages)


def test_rope_append_of_many_tokens():
    m = fa()
    T, hq, hkv, hd = 5003, 4, 2, 128
    q, k, v = torch.randn(T, hq + 2 * hkv, hd, device="cuda").bfloat16().split([hq, hkv, hkv], 1)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    table = m.rope_table(1e4 ** (-np.arange(64) / 64))
    slots = torch.randperm(T + 101, device="cuda")[:T].int()
    pages = [m.alloc_pages(5104 // 16, hkv, hd, 16).fill_(0) for _ in range(2)]
    q_out, q2, k2 = torch.empty_like(q), torch.empty_like(q), torch.empty(T, hkv, hd, device="cuda").bfloat16()
    m.rope_append(q, k, v, q_out, pos, table, slots, pages[0], page_rows=16)
    m.rope(q, k, q2, k2, pos, table)
    m.paged_append(k2, v, slots, pages[1], page_rows=16)
    assert torch.equal(q_out, q2) and torch.equal(*pages)


def test_rope_append_flags_bad_slots_and_tables():
    m = fa()
    rng = np.random.default_rng(1)
    q, k, v, pos, table, slots, pages = rope_case(rng, "bf16", 5, 2, 1, 64, 64, 1)
    before = pages.clone()
    for bad in (128, -2, 1 << 30):
        m.rope_append(q, k, v, torch.empty_like(q), pos, table, ints([bad] * 5), pages, page_rows=32)
        assert m.get_device_error() == m.ERR_DEVICE
    assert torch.equal(pages, before)
    table[3, 2] = 1  # an axis without positions
    m.rope_append(q, k, v, torch.empty_like(q), pos, table, ints([0, 1, 2, 3, 4]), pages, page_rows=32)
    assert m.get_device_error() == m.ERR_DEVICE


def test_rope_append_in_a_graph_on_another_stream():
    m = fa()
    rng = np.random.default_rng(2)
    q, k, v, pos, table, slots, pages = rope_case(rng, "f16", 20, 4, 2, 128, 128, 1)
    q_out, want, twin = torch.empty_like(q), torch.empty_like(q), pages.clone()
    m.rope_append(q, k, v, q_out, pos, table, slots, pages, page_rows=32)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.rope_append(q, k, v, q_out, pos, table, slots, pages, page_rows=32)
    for step in range(3):
        q.copy_(torch.randn_like(q))
        k.copy_(torch.randn_like(k))
        pos.add_(1)
        m.rope_append(q, k, v, want, pos, table, slots, twin, page_rows=32)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(q_out, want) and torch.equal(pages, twin)


# ---------------------------------------------------------------- all together

@pytest.mark.parametrize("cap,bias", [(0.0, False), (12.0, True)])
@pytest.mark.parametrize("hd", [64, 256])
def test_prompts_then_steps(hd, cap, bias):
    """Prompts go through packed attention while their rows enter the pages, then tokens follow one at a time:
    each step's attention over the pages is the row that packed attention gives for the whole document. K and V
    are values that 4-bit codes hold exactly, and the rotation is by no angle, so that both see the same numbers."""
    m = fa()
    hq, hkv, page_rows, steps = 4, 2, 16, 5
    lens = [40, 1, 133]
    R = len(lens)
    full = [n + steps for n in lens]
    g = torch.Generator("cuda").manual_seed(hd)
    q = torch.randn(sum(full), hq, hd, device="cuda", generator=g).bfloat16()

    def codes():  # sixteenths up to 8, a -8 or 8 in each block of 32 (the scale is of the largest)
        x = torch.randint(-7, 9, (sum(full), hkv, hd // 32, 32), device="cuda", generator=g)
        x[..., 0] = 8
        return (x.flatten(-2) / 8).bfloat16()
    k, v = codes(), codes()
    slopes = torch.tensor([0.5, 0.25, 0.1, 0.01], device="cuda") if bias else None
    cu = np.concatenate([[0], np.cumsum(full)])
    want = torch.empty_like(q)
    wlse = torch.empty(hq, q.shape[0], device="cuda")
    m.packed_attn(q, k, v, want, ints(cu), cap=cap, slopes=slopes, lse=wlse, workspace=torch.empty(
        m.packed_attn_workspace_bytes(R, q.shape[0], hq, hkv, hd), dtype=torch.uint8, device="cuda"))

    n_pages = 64
    pages = m.alloc_pages(n_pages, hkv, hd, page_rows)
    ring = ints(np.random.default_rng(1).permutation(n_pages))
    state, table = ints([0, n_pages, 0]), ints(np.full((R, 12), -1))
    rope = m.rope_table([0.0] * (hd // 2))
    ws = torch.empty(m.paged_attn_workspace_bytes(hd), dtype=torch.uint8, device="cuda")
    now = ints([0] * R)
    half, least = packed_ref.EPS[torch.bfloat16], 2.0 ** -24
    for step in range(steps + 1):
        fresh = lens if step == 0 else [1] * R
        first = [0 if step == 0 else n + step - 1 for n in lens]
        at = torch.cat([torch.arange(cu[r] + first[r], cu[r] + first[r] + fresh[r]) for r in range(R)]).cuda()
        T = at.numel()
        new, after = ints([0] * R), ints([0, 0, 0])
        cuq, slots, pos = ints([0] * (R + 1)), ints([0] * T), ints([0] * T)
        m.page_plan(now, ints(fresh), ring, state[:2].clone(), table, after, new, cuq, slots, pos, page_rows=page_rows)
        qs = q[at]
        m.rope_append(qs, k[at], v[at], qs, pos, rope, slots, pages, page_rows=page_rows)
        out, lse = torch.empty_like(qs), torch.empty(hq, T, device="cuda")
        m.paged_attn(qs, out, cuq, new, table, pages, n_kv_heads=hkv, page_rows=page_rows, cap=cap, slopes=slopes,
                     lse=lse, workspace=ws)
        # each side: weights rounded (2^-8 packed, 2^-10 paged) times values up to 1, and the result
        tol = (half + 2.0 ** -10) + 2 * half * want[at].double().abs() + least
        assert ((out.double() - want[at].double()).abs() <= tol).all(), step
        assert ((lse - wlse[:, at]).abs() <= 2.0 ** -20 * (hd + cap + 160)).all(), step
        state, now = after, new
    assert m.get_device_error() == m.OK


@pytest.mark.parametrize("hd", [64, 256])
def test_rotated_prompts_then_steps(hd):
    """What a server of a rotary model with capped scores runs: the prompts' heads are rotated (fa_rope), attend packed, and
    their rows enter the pages (fa_paged_append: packed attention wants the rotated k, which fa_rope_append keeps to
    itself); then tokens follow one at a time, rotated and appended in one call, and attend over the pages."""
    m = fa()
    hq, hkv, page_rows, steps, cap = 4, 2, 16, 4, 12.0
    lens = [40, 1, 133]
    R = len(lens)
    full = [n + steps for n in lens]
    cu = np.concatenate([[0], np.cumsum(full)])
    g = torch.Generator("cuda").manual_seed(hd)
    q, k, v = torch.randn(sum(full), hq + 2 * hkv, hd, device="cuda", generator=g).bfloat16().split([hq, hkv, hkv], 1)
    rope = m.rope_table(1e4 ** (-np.arange(hd // 2) / (hd // 2)))
    qr, kr = torch.empty_like(q), torch.empty_like(k)
    m.rope(q, k, qr, kr, ints(np.concatenate([np.arange(n) for n in full])), rope)
    # what the pages hold of each request's rows
    held = [[ref.decode(*ref.encode(x[cu[r]:cu[r + 1]].float().cpu().numpy())) for x in (kr, v)] for r in range(R)]
    slopes = np.array([0.5, 0.25, 0.1, 0.01], np.float32)
    bias = torch.from_numpy(slopes).cuda()

    n_pages = 64
    pages = m.alloc_pages(n_pages, hkv, hd, page_rows)
    ring = ints(np.random.default_rng(1).permutation(n_pages))
    state, table = ints([0, n_pages, 0]), ints(np.full((R, 12), -1))
    ws = torch.empty(m.paged_attn_workspace_bytes(hd), dtype=torch.uint8, device="cuda")
    now = ints([0] * R)
    for step in range(steps + 1):
        fresh = lens if step == 0 else [1] * R
        first = [0 if step == 0 else n + step - 1 for n in lens]
        at = torch.cat([torch.arange(cu[r] + first[r], cu[r] + first[r] + fresh[r]) for r in range(R)]).cuda()
        T = at.numel()
        new, after = ints([0] * R), ints([0, 0, 0])
        cuq, slots, pos = ints([0] * (R + 1)), ints([0] * T), ints([0] * T)
        m.page_plan(now, ints(fresh), ring, state[:2].clone(), table, after, new, cuq, slots, pos, page_rows=page_rows)
        qs, ks, vs = q[at], k[at], v[at]
        out, lse = torch.empty_like(qs), torch.empty(hq, T, device="cuda")
        if step == 0:
            m.rope(qs, ks, qs, ks, pos, rope)
            m.packed_attn(qs, ks, vs, out, cuq, cap=cap, slopes=bias, lse=lse, workspace=torch.empty(
                m.packed_attn_workspace_bytes(R, T, hq, hkv, hd), dtype=torch.uint8, device="cuda"))
            m.paged_append(ks, vs, slots, pages, page_rows=page_rows)
            assert torch.equal(qs, qr[at]) and torch.equal(ks, kr[at])
            want = packed_ref.packed(qs, ks, vs, cuq.tolist(), slopes=bias, cap=cap)
            assert ((out.double() - want["out"]).abs() <= want["out_err"]).all()
            assert ((lse.double() - want["lse"]).abs() <= want["lse_err"]).all()
        else:
            m.rope_append(qs, ks, vs, qs, pos, rope, slots, pages, page_rows=page_rows)
            assert torch.equal(qs, qr[at])
            m.paged_attn(qs, out, cuq, new, table, pages, n_kv_heads=hkv, page_rows=page_rows, cap=cap, slopes=bias,
                         lse=lse, workspace=ws)
            for r in range(R):
                n = first[r] + 1
                kp, vp = (x[:n] for x in held[r])
                want, wlse, size, off, codes = attend(qs[r:r + 1].double().cpu().numpy(), n - 1, kp, vp, cap, slopes, 0, 0,
                                                      1 / math.sqrt(hd))
                # the bounds of run_paged for bf16
                ds = off * 2.0 ** -21 + cap * 2.0 ** -21
                block = np.abs(vp).reshape(n, hkv, hd // 32, 32).max(-1) / 7
                block = np.repeat(np.repeat(block, 32, -1), hq // hkv, 1).max(0)
                tol = size * (2.0 ** -10 * (1 + 2.0 ** -11) + 2 * ds.T[:, :, None]) + 2.0 ** -24
                tol = tol + 2 * (-(-n // 16) + 40) * 2.0 ** -23 * 16 * block
                tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
                assert (np.abs(out[r:r + 1].double().cpu().numpy() - want) <= tol).all(), (step, r)
                ds = ds + codes * 2.0 ** -21
                assert (np.abs(lse[:, r:r + 1].double().cpu().numpy() - wlse) <= ds + 2.0 ** -21).all(), (step, r)
        state, now = after, new
    assert m.get_device_error() == m.OK
