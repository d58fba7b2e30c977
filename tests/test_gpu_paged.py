"""Paged serving on the GPU against the definition in 64 bits (paged_ref.py)."""
import math

import numpy as np
import pytest
import torch

import paged_ref as ref
from gpu_util import POISON_BYTE, check_guards, fa, guarded

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def ints(a):
    a = np.asarray(a, np.int32)
    t = guarded(a.shape, torch.int32)
    t.copy_(torch.from_numpy(a))
    return t


def on_gpu(x, dtype, spare=0):
    """float64 numpy -> the GPU in a type; spare: values between the rows of dim 0 (a strided tensor)."""
    x = ref.round_type(x, dtype)
    if not spare:
        return torch.from_numpy(x).to(DT[dtype]).cuda(), x
    row = int(np.prod(x.shape[1:]))
    wide = torch.full((x.shape[0], row + spare), float("nan"), dtype=DT[dtype], device="cuda")
    t = wide[:, :row].unflatten(1, x.shape[1:])
    t.copy_(torch.from_numpy(x))
    return t, x


def host(t):
    return t.detach().double().cpu().numpy()


# --------------------------------------------------------------------- plan

def random_step(rng, n_reqs, page_rows, max_pages, n_pages, most_fresh, short=0):
    """A consistent state: lengths, a ring in the middle of its life, a table."""
    most = max_pages * page_rows
    fresh = np.where(rng.random(n_reqs) < 0.3, rng.integers(0, most_fresh + 1, n_reqs), 1)
    fresh = np.where(rng.random(n_reqs) < 0.15, -1, np.minimum(fresh, most))
    cached = np.minimum(rng.integers(0, most + 1, n_reqs), most - np.maximum(fresh, 0))
    used = -(-cached // page_rows)
    order = rng.permutation(n_pages)
    assert used.sum() <= n_pages
    table = np.full((n_reqs, max_pages), -1)
    at = 0
    for r in range(n_reqs):
        table[r, :used[r]] = order[at:at + used[r]]
        at += used[r]
    free = order[at:len(order) - short] if short else order[at:]
    head = int(rng.integers(n_pages))
    ring = np.full(n_pages, -7)
    ring[(head + np.arange(len(free))) % n_pages] = free
    return cached, fresh, ring, [head, len(free)], table


def run_plan(cached, fresh, ring, state, table, page_rows, max_tokens):
    m = fa()
    R = len(cached)
    t = dict(cached=ints(cached), fresh=ints(fresh), free_ring=ints(ring), ring_state=ints(state),
             block_table=ints(table), ring_state_out=ints([-9] * 3), seq_lens=ints([-9] * R),
             cu_fresh=ints([-9] * (R + 1)), slot_map=ints([-9] * max_tokens),
             positions=ints([-9] * max_tokens))
    m.page_plan(*t.values(), page_rows=page_rows)
    torch.cuda.synchronize()
    check_guards(*t.items())
    return t, dict(ring=t["free_ring"].tolist(), table=t["block_table"].tolist(), lens=t["seq_lens"].tolist(),
                   cu=t["cu_fresh"].tolist(), slots=t["slot_map"].tolist(),
                   positions=t["positions"].tolist(), state=t["ring_state_out"].tolist())


@pytest.mark.parametrize("n_reqs,page_rows,max_pages,most_fresh,pad", [
    (1, 16, 1, 16, 0), (1, 256, 3, 700, 9), (2, 16, 4, 3, 1), (33, 32, 5, 100, 0), (511, 16, 9, 40, 3),
    (513, 64, 4, 90, 2), (1025, 128, 3, 11, 70), (5000, 16, 3, 30, 1)])
def test_plan(n_reqs, page_rows, max_pages, most_fresh, pad):
    rng = np.random.default_rng(n_reqs)
    step = random_step(rng, n_reqs, page_rows, max_pages, n_reqs * max_pages + 3, most_fresh)
    tokens = int(np.maximum(step[1], 0).sum()) + pad
    _, got = run_plan(*step, page_rows, tokens)
    want = ref.plan(*step, page_rows, tokens)
    for name in want:
        assert got[name] == [list(map(int, x)) if name == "table" else int(x) for x in want[name]], name
    assert fa().get_device_error() == fa().OK


def test_plan_with_too_few_pages_gives_them_in_order():
    rng = np.random.default_rng(3)
    for n_free in (0, 1, 5, 17):
        cached = np.array([0, 16, 3, 31, 32, 7, 0, 64])
        fresh = np.array([20, 1, 2, 1, 33, -1, 0, 1])
        used = -(-cached // 16)
        order = rng.permutation(40)
        table, at = np.full((8, 6), -1), 0
        for r in range(8):
            table[r, :used[r]] = order[at:at + used[r]]
            at += used[r]
        ring = np.full(40, -7)
        ring[(38 + np.arange(n_free)) % 40] = order[at:at + n_free]
        step = (cached, fresh, ring, [38, n_free], table)
        _, got = run_plan(*step, 16, 60)
        want = ref.plan(*step, 16, 60)
        for name in want:
            assert got[name] == [list(map(int, x)) if name == "table" else int(x) for x in want[name]], (n_free, name)
        assert fa().get_device_error() == fa().OK


def test_plan_flags_bad_device_data_and_stays_in_bounds():
    m = fa()
    good = ([3, 20], [1, 1], [5, 4, 3, 2, 1, 0], [0, 3], [[0, -1], [1, 2]])

    def flagged(cached=None, fresh=None, ring=None, state=None, table=None, tokens=4):
        step = [x if y is None else y for x, y in zip(good, (cached, fresh, ring, state, table))]
        _, got = run_plan(*step, 16, tokens)
        assert m.get_device_error() == m.ERR_DEVICE
        return got

    got = flagged(cached=[-1, 20])
    assert got["lens"] == [0, 21] and got["slots"] == [-1, 2 * 16 + 4, -1, -1] and got["cu"] == [0, 1, 2]
    got = flagged(fresh=[30, 1], tokens=32)               # more rows than the table has pages for
    assert got["lens"] == [0, 21] and got["slots"][:30] == [-1] * 30 and got["slots"][30] == 36
    got = flagged(fresh=[1 << 30, 1])                     # and more tokens than there is room for
    assert got["cu"] == [0, 4, 4] and got["slots"] == [-1] * 4
    got = flagged(fresh=[-2, 1])
    assert got["lens"] == [0, 21] and got["cu"] == [0, 0, 1]
    for state in ([-1, 3], [6, 3], [0, 7], [0, -1]):
        got = flagged(state=state, fresh=[14, -1], tokens=14)
        assert got["lens"] == [3, 0] and got["state"][1] == 0 and got["state"][2] == 1
        assert got["ring"] == good[2]
    got = flagged(table=[[6, -1], [1, -1]])               # pages out of range under fresh tokens
    assert got["slots"] == [-1] * 4 and got["lens"] == [4, 21]
    got = flagged(state=[0, 5], fresh=[-1, -1])           # more pages back than the ring has room for
    assert got["state"][1] == 6 and sorted(got["ring"][:5]) == [1, 2, 3, 4, 5] and got["ring"][5] == 0
    got = flagged(tokens=1)                               # two tokens, room for one
    assert got["cu"] == [0, 1, 1] and got["slots"] == [3]


def test_plan_refuses_shapes():
    m = fa()
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    args = [z(2), z(2), z(8), z(2), z(2, 3), z(3), z(2), z(3), z(4), z(4)]
    for i, bad in ((1, z(3)), (3, z(3)), (4, z(3, 3)), (4, z(6)), (5, z(2)), (7, z(2)), (9, z(5)),
                   (0, z(2).long()), (2, z(16)[::2]), (6, z(2).cpu())):
        with pytest.raises(ValueError):
            m.page_plan(*[bad if j == i else a for j, a in enumerate(args)], page_rows=16)


# --------------------------------------------------------------------- rope

@pytest.mark.parametrize("dtype", ("f32", "f16", "bf16"))
@pytest.mark.parametrize("T,hq,hkv,hd,rd,sections,interleaved,adjacent,inverse,spare", [
    (1, 1, 1, 64, 64, [32], False, False, False, 0),
    (7, 8, 2, 64, 32, [16], False, True, False, 64),
    (33, 16, 2, 256, 64, [12, 10, 10], True, False, True, 512),
    (130, 4, 4, 128, 128, [16, 24, 24], False, False, False, 0),
    (5, 3, 1, 96, 96, [24, 8, 8, 8], True, True, True, 8),
    (3, 5, 0, 80, 20, [10], False, False, False, 3),      # nothing a multiple of 16 bytes
    (2, 0, 3, 7, 6, [2, 1], False, True, True, 1),
    (1000, 32, 8, 128, 128, [64], False, True, False, 0)])
def test_rope(dtype, T, hq, hkv, hd, rd, sections, interleaved, adjacent, inverse, spare):
    m = fa()
    rng = np.random.default_rng(T * hd + rd)
    half = rd // 2
    freq = 1e4 ** (-np.arange(half) / half)
    freq[0] = 1.0
    # near positions, far ones and negative ones
    pos = rng.integers(0, 5000, (len(sections), T))
    pos[0, :: 3] = rng.integers(2 ** 30, 2 ** 31 - 1, len(pos[0, ::3]))
    pos[-1, 1::3] = -rng.integers(0, 2 ** 31 - 1, len(pos[-1, 1::3]))
    axis = ref.axes_of(half, sections, interleaved)
    table = m.rope_table(freq, sections, interleaved=interleaved)
    pairs = []
    for heads in (hq, hkv):
        if heads == 0:
            pairs.append((None, None, None))
            continue
        x, exact = on_gpu(rng.standard_normal((T, heads, hd)) * 3, dtype, spare)
        pairs.append((x, guarded((T, heads, hd), DT[dtype], fill=float("nan")), exact))
    (q, qo, qx), (k, ko, kx) = pairs
    m.rope(q, k, qo, ko, ints(pos), table, adjacent=adjacent, inverse=inverse)
    for x, y, exact in pairs:
        if x is None:
            continue
        check_guards(("out", y))
        want = ref.rope(exact, pos, freq, axis, adjacent, inverse)
        # In turns the angle is off by at most 2^-33 (32 bits kept, rounded), by |pos| (2^-64 + f 2^-53) through
        # its table entry, and by 2^-26 where it becomes an fp32 argument; times 2 pi. The 64-bit reference's own
        # |pos| f 2^-53 comes on top. sincospif is off by 2 steps (2^-23), two products and a sum by 2^-23 of |x| + |y|.
        f = freq / (2 * math.pi)
        angle = 2 * math.pi * (2.0 ** -33 + 2.0 ** -26 + np.abs(pos[axis, :]).T * (2.0 ** -64 + 2 * f * 2.0 ** -53))
        i = np.arange(half)
        lo, hi = (2 * i, 2 * i + 1) if adjacent else (i, i + half)
        size = np.zeros_like(exact)
        size[..., lo] = size[..., hi] = np.abs(exact[..., lo]) + np.abs(exact[..., hi])
        slack = np.zeros_like(exact)
        slack[..., lo] = slack[..., hi] = (angle + 2.0 ** -23 + 2.0 ** -23)[:, None, :]
        tol = size * slack
        tol += ref.HALF_STEP[dtype] * (np.abs(want) + tol) * (size > 0) + 2.0 ** -25 * (dtype == "f16")
        assert np.all(np.abs(host(y) - want) <= tol)
        assert np.array_equal(host(y)[..., rd:], exact[..., rd:])
        # in place: the same bits
        z = x.clone()
        m.rope(*((z, None, z, None) if x is q else (None, z, None, z)), ints(pos), table, adjacent=adjacent,
               inverse=inverse)
        assert torch.equal(z, y)


def test_rope_inverse_is_the_gradient():
    """The inverse rotation of g is the gradient of <g, rope(x)>: against differences, and it undoes the rotation."""
    m = fa()
    rng = np.random.default_rng(9)
    T, H, hd = 6, 3, 64
    table = m.rope_table(1e4 ** (-np.arange(32) / 32), [12, 10, 10], interleaved=True)
    pos = ints(rng.integers(0, 900, (3, T)))
    x, g = (torch.from_numpy(rng.standard_normal((T, H, hd)).astype(np.float32)).cuda() for _ in range(2))
    grad, y = torch.empty_like(g), torch.empty_like(x)
    m.rope(g, None, grad, None, pos, table, inverse=True)

    def loss(v):
        m.rope(v, None, y, None, pos, table)
        return float((y.double() * g.double()).sum())

    for t, h, e in rng.integers(0, [T, H, hd], (12, 3)):
        up, down = x.clone(), x.clone()
        up[t, h, e] += 0.5
        down[t, h, e] -= 0.5
        # linear in x: the difference over a step of 1 has fp32 rounding alone, 2^-22 of the two rotated values
        # (|x| + 1 and |g| at most 5 here) in each of the two losses
        assert abs(loss(up) - loss(down) - float(grad[t, h, e])) <= 2 * 2 * 6 * 5 * 2.0 ** -22
    m.rope(x, None, y, None, pos, table)
    m.rope(y, None, y, None, pos, table, inverse=True)
    assert float((y - x).abs().max()) <= 5 * 2 * 2 * 2.0 ** -21


def test_rope_refuses():
    m = fa()
    table = m.rope_table([1.0] * 16)
    x = torch.zeros(4, 2, 32, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in (lambda: m.rope(None, None, None, None, pos, table),
                lambda: m.rope(x, None, None, None, pos, table),
                lambda: m.rope(x, x.half(), x, x.half(), pos, table),
                lambda: m.rope(x, None, x[:, :1], None, pos, table),
                lambda: m.rope(x, None, x, None, pos[:3], table),
                lambda: m.rope(x, None, x, None, pos.long(), table),
                lambda: m.rope(x.transpose(0, 1), None, x.transpose(0, 1), None, pos, table),
                lambda: m.rope(x, None, x, None, pos, table[:, :3]),
                lambda: m.rope(x.double(), None, x.double(), None, pos, table),
                lambda: m.rope(x.cpu(), None, x.cpu(), None, pos, table)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(m.FAError):  # more rotated dims than a head has
        m.rope(x, None, x, None, pos, m.rope_table([1.0] * 17))


# ------------------------------------------------------------ append, gather

def pool_of(m, n_pages, hkv, hd, page_rows):
    """Pages of 0xff bytes: NaN scales and factors wherever nothing was written."""
    return guarded(n_pages * m.page_bytes(hkv, hd, page_rows), torch.uint8, fill_byte=POISON_BYTE)


def append(m, pages, k, v, slots, page_rows):
    m.paged_append(k, v, ints(slots), pages, page_rows=page_rows)


@pytest.mark.parametrize("dtype", ("f32", "f16", "bf16"))
@pytest.mark.parametrize("hd,hkv,page_rows,T,spare", [
    (64, 1, 16, 1, 0), (64, 3, 32, 37, 128), (128, 2, 16, 50, 0), (256, 2, 64, 19, 64), (256, 1, 256, 70, 0)])
def test_append_bytes(dtype, hd, hkv, page_rows, T, spare):
    """Every byte of the pages: rows in scattered slots, the rest as it was."""
    m = fa()
    rng = np.random.default_rng(hd + T)
    n_pages = 2 * T // page_rows + 3
    pages = pool_of(m, n_pages, hkv, hd, page_rows)
    slots = rng.permutation(n_pages * page_rows)[:T]
    if T > 4:
        slots[3] = -1  # a padded token
    x = rng.standard_normal((2, T, hkv, hd))
    x[0, 0, 0, :32] = 0                                   # an empty block
    x[1, T // 2] = 0                                      # an empty row
    x[0, T // 2] *= 300
    x[1, T - 1, :, 32:] *= 1e-4                           # blocks far below the row's largest
    k, kx = on_gpu(x[0], dtype, spare)
    v, vx = on_gpu(x[1], dtype, 2 * spare)
    append(m, pages, k, v, slots, page_rows)
    torch.cuda.synchronize()
    check_guards(("pages", pages))
    want = np.full(pages.numel(), POISON_BYTE, np.uint8)
    for t, slot in enumerate(slots):
        for h in range(hkv):
            if slot >= 0:
                ref.put_row(want, page_rows, hkv, hd, int(slot), h, kx[t, h], 0)
                ref.put_row(want, page_rows, hkv, hd, int(slot), h, vx[t, h], 1)
    assert np.array_equal(pages.cpu().numpy(), want)
    assert m.get_device_error() == m.OK


def test_append_any_magnitude_and_values_without_one():
    """Rows of 1e-30 and 1e30, of infinities and NaN: the factor keeps the first, the others stay in their row."""
    m = fa()
    hd, rng = 64, np.random.default_rng(1)
    x = rng.standard_normal((6, 1, hd)).astype(np.float32)
    x[0] *= np.float32(1e-30)
    x[1] *= np.float32(1e30)
    x[2] *= np.float32(1e-42)                             # below fp32's normal range
    x[3, 0, 5] = np.inf
    x[4, 0, 40] = np.nan
    pages = pool_of(m, 1, 1, hd, 16)
    t = torch.from_numpy(x).cuda()
    append(m, pages, t, t, range(6), 16)
    got = pages.cpu().numpy()
    want = np.full_like(got, POISON_BYTE)
    for r in (0, 1, 5):
        ref.put_row(want, 16, 1, hd, r, 0, x[r, 0], 0)
        ref.put_row(want, 16, 1, hd, r, 0, x[r, 0], 1)
    for r in (0, 1, 5):
        for v in (0, 1):
            base = v * (9 * hd + 32)
            places = [base + ref.code_place(hd, r, e, v)[0] for e in range(hd)]
            places += [base + ref.scale_place(hd, r, b, v) + i for b in range(2) for i in (0, 1)]
            places += [base + 9 * hd + 2 * r, base + 9 * hd + 2 * r + 1]
            assert np.array_equal(got[places], want[places])


@pytest.mark.parametrize("hd", (64, 128, 256))
def test_append_bytes_of_odd_rows(hd):
    """Subnormal and largest values, ties, NaN and infinities anywhere: codes as Q4_0's encoder defines them (amax
    ignores NaN; a NaN product is 0, products beyond the codes are clamped), scales and factors of the same amax."""
    m = fa()
    rng = np.random.default_rng(hd)
    T = 320
    x = (rng.standard_normal((T, hd // 32, 32)) * 10.0 ** rng.uniform(-46, 37, (T, 1, 1))
         * 10.0 ** rng.uniform(-3, 0, (T, hd // 32, 1))).astype(np.float32)
    ties = rng.integers(-16, 16, x.shape).astype(np.float32) / 2
    ties[..., 0] = -8
    x[:40] = ties[:40] * np.exp2(rng.integers(-140, 120, (40, 1, 1))).astype(np.float32)
    for rows, value in ((range(40, 80), np.nan), (range(70, 100), np.inf), (range(100, 120), -np.inf),
                        (range(120, 140), np.finfo(np.float32).max), (range(140, 160), 2.0 ** -149), (range(150, 180), 0)):
        for r in rows:
            x[r][rng.random(x[r].shape) < rng.choice([0.02, 0.3, 1.0])] = value
    with np.errstate(all="ignore"):
        d = np.fmax.reduce(np.abs(x), -1, initial=0) / np.float32(-8)
        inv = np.where(d != 0, np.float32(1) / np.where(d != 0, d, np.float32(1)), np.float32(0)).astype(np.float32)
        p = (x * inv[..., None]).astype(np.float32)
        codes = np.clip(np.rint(np.where(np.isnan(p), 0, p)), -8, 7) + 8
        top = np.abs(d).max(-1)
        e = np.where(np.isinf(top), 127, np.clip(np.frexp(np.where((top > 0) & ~np.isinf(top), top, 1))[1] - 1, -126, 127))
        factors = np.where(top > 0, np.exp2(e.astype(np.float64)), 1.0).astype(np.float32)
        scales = (d / factors[:, None]).astype(np.float16)
    pages = pool_of(m, T // 16, 1, hd, 16)
    t = torch.from_numpy(x.reshape(T, 1, hd)).cuda()
    append(m, pages, t, t, range(T), 16)
    got = pages.cpu().numpy().reshape(T // 16, 2, -1)
    for v in (0, 1):
        places = [ref.code_place(hd, r, i, v) for r in range(16) for i in range(hd)]
        at, shift = (np.array(a).reshape(16, hd) for a in zip(*places))
        assert np.array_equal((got[:, v][:, at] >> shift & 15).reshape(T, hd), codes.reshape(T, hd))
        at = np.array([[ref.scale_place(hd, r, b, v) for b in range(hd // 32)] for r in range(16)])
        have = (got[:, v][:, at] | got[:, v][:, at + 1].astype(np.uint16) << 8).reshape(T, -1)
        assert np.array_equal(have, scales.view(np.uint16))
        at = 9 * hd + 2 * np.arange(16)
        have = (got[:, v][:, at] | got[:, v][:, at + 1].astype(np.uint32) << 8).reshape(T)
        assert np.array_equal(have << 16, factors.view(np.uint32))
    assert m.get_device_error() == m.OK


def test_append_slots_out_of_range():
    m = fa()
    pages = pool_of(m, 2, 1, 64, 16)
    x = torch.randn(5, 1, 64, device="cuda")
    append(m, pages, x, x, [-1, 32, -2, 2 ** 31 - 1, -2 ** 31], 16)
    torch.cuda.synchronize()
    check_guards(("pages", pages))
    assert bool((pages == POISON_BYTE).all())
    assert m.get_device_error() == m.ERR_DEVICE
    append(m, pages, x[:1], x[:1], [-1], 16)
    assert m.get_device_error() == m.OK


def filled(m, rng, lens, hkv, hd, page_rows, spare_pages=2, k_size=1.0, v_size=1.0):
    """A pool with one request for each length, filled by appends in random pages.
    Returns pages, table (numpy, -1 past the rows), and each request's K, V as the values they stand for."""
    used = [-(-L // page_rows) for L in lens]
    n_pages = sum(used) + spare_pages
    order = rng.permutation(n_pages)
    table = np.full((len(lens), max(1, max(used))), -1)
    at, slots, ks, vs = 0, [], [], []
    for r, L in enumerate(lens):
        table[r, :used[r]] = order[at:at + used[r]]
        at += used[r]
        p = np.arange(L)
        slots.append(table[r, p // page_rows] * page_rows + p % page_rows)
        ks.append((rng.standard_normal((L, hkv, hd)) * k_size).astype(np.float32))
        vs.append((rng.standard_normal((L, hkv, hd)) * v_size).astype(np.float32))
    pages = pool_of(m, n_pages, hkv, hd, page_rows)
    if at:
        append(m, pages, torch.from_numpy(np.concatenate(ks)).cuda(), torch.from_numpy(np.concatenate(vs)).cuda(),
               np.concatenate(slots), page_rows)
    return pages, table, [ref.decode(*ref.encode(k)) for k in ks], [ref.decode(*ref.encode(v)) for v in vs]


@pytest.mark.parametrize("hd,hkv,page_rows,lens", [
    (64, 2, 16, [1, 0, 16, 17, 100]), (128, 3, 64, [63, 64, 65]), (256, 2, 256, [500]), (256, 1, 32, [31, 0, 33])])
def test_gather_bits(hd, hkv, page_rows, lens):
    """The planes hold the rows' values rounded to binary16, bit for bit; other rows stay as they were."""
    m = fa()
    pages, table, ks, vs = filled(m, np.random.default_rng(hd), lens, hkv, hd, page_rows)
    max_seq = max(lens) + 5
    pb = m.kv_plane_bytes(m.KV_F16, hkv, max_seq, hd)
    kp, vp = (guarded(len(lens) * pb, torch.uint8, fill_byte=POISON_BYTE) for _ in range(2))
    m.paged_gather(pages, ints(table), ints(lens), kp, vp, n_kv_heads=hkv, head_dim=hd, page_rows=page_rows,
                   max_seq=max_seq)
    assert m.get_device_error() == m.OK
    check_guards(("k", kp), ("v", vp))
    for planes, want in ((kp, ks), (vp, vs)):
        got = planes.cpu().numpy().reshape(len(lens), pb)
        for r, L in enumerate(lens):
            rows = got[r][:hkv * max_seq * hd * 2].reshape(hkv, max_seq, hd * 2)
            x = np.ascontiguousarray(want[r].astype(np.float16).transpose(1, 0, 2)).view(np.uint8)
            assert np.array_equal(rows[:, :L], x.reshape(hkv, L, hd * 2))
            assert np.all(rows[:, L:] == POISON_BYTE) and np.all(got[r][hkv * max_seq * hd * 2:] == POISON_BYTE)


def test_gather_flags_lengths_and_pages():
    m = fa()
    hd, hkv, P, max_seq = 64, 1, 16, 40
    pages, table, ks, _ = filled(m, np.random.default_rng(2), [32, 32, 32], hkv, hd, P)
    pb = m.kv_plane_bytes(m.KV_F16, hkv, max_seq, hd)
    kp, vp = (guarded(3 * pb, torch.uint8, fill_byte=POISON_BYTE) for _ in range(2))
    table[2, 0] = 99
    m.paged_gather(pages, ints(table), ints([-4, 33, 32]), kp, vp, n_kv_heads=hkv, head_dim=hd, page_rows=P,
                   max_seq=max_seq)
    assert m.get_device_error() == m.ERR_DEVICE
    check_guards(("k", kp), ("v", vp))
    got = kp.cpu().numpy().reshape(3, pb)[:, :max_seq * hd * 2].reshape(3, max_seq, hd * 2)
    assert np.all(got[0] == POISON_BYTE) and np.all(got[1, 32:] == POISON_BYTE)
    assert np.all(got[2, :16] == POISON_BYTE) and np.all(got[2, 32:] == POISON_BYTE)
    for r, lo in ((1, 0), (2, 16)):
        assert np.array_equal(got[r, lo:32], ks[r][lo:32, 0].astype(np.float16).view(np.uint8).reshape(32 - lo, -1))


# ---------------------------------------------------------------- attention

def attn_bounds(q, k, v, dtype, scale):
    """How far out and lse may be off, from the kernel's arithmetic: per (query, head).

    Scores. A block's products are summed in fp32 with the codes 0..15 (their offset 8 is subtracted by the sum's
    start), so a term is at most 15 |q| + 8 |q| code steps; every sum in the tensor core may lose a step (2^-23) in
    each of 4 additions, and the blocks' sums and the scale another 2^-23 each. With B = sum over dims of 23 |q| |s|
    the score is off by (4 + 2) 2^-23 B; the pair of binary16 terms of an fp32 q adds 2^-22 B (one term is exact
    for f16 and bf16 queries). The exponential adds 2^-22 + |score| 2^-23 <= 2^-22 + 2^-23 B.
    Weights: rounded twice to binary16 (2 * 2^-11) for bf16, to a pair of terms (2^-20) otherwise. V codes enter
    with their offset: sums of 16 w |s| at most, 2^-23 lost in each addition of 16 rows, and the sum of weights too.
    """
    g = q.shape[1] // k.shape[1]
    step = lambda x: np.repeat(np.abs(x).reshape(*x.shape[:2], x.shape[2] // 32, 32).max(-1) / 7, 32, -1)  # noqa: E731
    kb, vb = step(k), step(v)
    B = 23 * scale * np.einsum("nhd,jhd->nhj", np.abs(q), np.repeat(kb, g, 1)).max(-1) if len(k) else np.zeros(q.shape[:2])
    d = 2.0 ** -23 * (8 + 1) * B + 2.0 ** -21
    eps = 2 * 2.0 ** -11 if dtype == "bf16" else 2.0 ** -20
    n = -(-len(k) // 16) + 40
    top = 16 * np.repeat(vb, g, 1).max(0) if len(k) else np.zeros(q.shape[1:])
    return (2 * d + eps + 2 * n * 2.0 ** -23)[..., None] * top, d + n * 2.0 ** -23 + 2.0 ** -22


def check_attn(lens, nqs, hq, hkv, hd, page_rows, dtype, *, sink=0, win=0, scale=0.0, spare=0, pad=0, k_size=1.0,
               v_size=1.0, q_size=1.0, drop=True, seed=0, extra_pages=2):
    """One call against the reference; returns the largest out and lse errors over their bounds."""
    m = fa()
    rng = np.random.default_rng(seed + 7 * hd + len(lens))
    pages, table, ks, vs = filled(m, rng, lens, hkv, hd, page_rows, k_size=k_size, v_size=v_size,
                                  spare_pages=extra_pages)
    if win > 0 and drop:  # pages that no query attends are gone
        for r, (L, n) in enumerate(zip(lens, nqs)):
            for i in range(-(-L // page_rows)):
                if i * page_rows >= sink and (i + 1) * page_rows - 1 < L - n - win + 1:
                    table[r, i] = -1
    T = sum(nqs)
    q, qx = on_gpu(rng.standard_normal((T + pad, hq, hd)) * q_size, dtype, spare)
    if spare:
        out = torch.full((T + pad, hq * hd + spare), 7.0, dtype=DT[dtype], device="cuda")
        o = out[:, :hq * hd].unflatten(1, (hq, hd))
    else:
        o = guarded((T + pad, hq, hd), DT[dtype], fill=7.0)
    lse = guarded((hq, T + pad), torch.float32, fill=7.0)
    ws = guarded(m.paged_attn_workspace_bytes(hd), torch.uint8, fill_byte=POISON_BYTE)
    cu = np.concatenate([[0], np.cumsum(nqs)])
    m.paged_attn(q, o, ints(cu), ints(lens), ints(table), pages, n_kv_heads=hkv, page_rows=page_rows, sink=sink,
                 win=win, scale=scale, lse=lse, workspace=ws)
    assert m.get_device_error() == m.OK
    check_guards(("lse", lse), ("workspace", ws))
    if spare:
        assert bool((out[:, hq * hd:] == 7.0).all())
    else:
        check_guards(("out", o))
    got, gl = host(o), host(lse)
    assert np.all(got[T:] == 7.0) and np.all(gl[:, T:] == 7.0)  # padding is left as it was
    sc = scale or 1 / math.sqrt(hd)
    num = den = 0.0
    for r, (L, n) in enumerate(zip(lens, nqs)):
        if n == 0:
            continue
        t = slice(cu[r], cu[r + 1])
        want, wl = ref.attend(qx[t], L, ks[r], vs[r], L - n, sink, win, sc)
        tol, ltol = attn_bounds(qx[t], ks[r], vs[r], dtype, sc)
        tol = tol + ref.HALF_STEP[dtype] * (np.abs(want) + tol) + (2.0 ** -25 if dtype == "f16" else 0.0)
        assert np.all(np.isfinite(got[t]))
        assert np.all(np.abs(got[t] - want) <= tol), f"request {r}: {np.max(np.abs(got[t] - want) / tol)}"
        dead = wl == -math.inf
        assert np.array_equal(gl[:, t] == -math.inf, dead) and np.all(got[t].transpose(1, 0, 2)[dead] == 0)
        ltol = ltol.T + np.abs(np.where(dead, 0, wl)) * 2.0 ** -22
        assert np.all(np.abs(gl[:, t][~dead] - wl[~dead]) <= ltol[~dead])
        num, den = num + ((got[t] - want) ** 2).sum(), den + (want ** 2).sum()
    if den:
        # Roundings are independent, so the 2-norm stays below half a step of the type; fp32's sums of a few
        # hundred terms stay below 2^-17. Binary16 below its normal range has steps of 2^-24 however small the
        # value is: half a step, 2^-25, for each of the T * hq * hd outputs.
        floor = 2.0 ** -25 * math.sqrt(T * hq * hd) if dtype == "f16" else 0.0
        assert math.sqrt(num) <= {"f32": 2.0 ** -17, "f16": 2.0 ** -10, "bf16": 2.0 ** -8}[dtype] * math.sqrt(den) + floor
    return q, o, lse


SHAPES = [
    # lens, queries, hq, hkv, hd, page_rows, sink, win
    ([1], [1], 1, 1, 64, 16, 0, 0),
    ([600], [1], 8, 2, 64, 16, 0, 0),
    ([15, 16, 17, 0, 33], [1, 1, 1, 1, 1], 16, 2, 256, 16, 0, 0),
    ([300, 5, 1000, 64], [1, 0, 1, 1], 16, 2, 256, 64, 0, 0),
    ([200, 3, 77], [5, 3, 2], 32, 8, 128, 32, 0, 0),
    ([2, 130], [4, 7], 16, 1, 128, 128, 0, 0),            # more queries than rows; groups of 16
    ([90, 500], [9, 1], 4, 4, 128, 256, 0, 0),            # heads that share nothing
    ([40, 700], [3, 2], 4, 2, 64, 16, 0, 0),
    ([500, 90, 40], [1, 2, 3], 8, 2, 256, 32, 4, 100),
    ([1000, 30], [2, 1], 8, 1, 64, 16, 37, 61),
    ([400], [3], 2, 2, 128, 16, 0, 1),
    ([700, 20, 0, 260], [1, 1, 1, 1], 4, 1, 128, 64, 500, 3),
]


@pytest.mark.parametrize("dtype", ("f32", "f16", "bf16"))
@pytest.mark.parametrize("case", SHAPES, ids=lambda c: f"h{c[2]}x{c[3]}d{c[4]}p{c[5]}w{c[7]}n{len(c[0])}")
def test_attn(case, dtype):
    lens, nqs, hq, hkv, hd, page_rows, sink, win = case
    check_attn(lens, nqs, hq, hkv, hd, page_rows, dtype, sink=sink, win=win)


@pytest.mark.parametrize("hd", (64, 128, 256))
def test_attn_strides_padding_and_scale(hd):
    check_attn([100, 31], [2, 1], 8, 2, hd, 16, "bf16", spare=3 * hd, pad=3, scale=0.3)
    check_attn([100, 31], [2, 1], 8, 2, hd, 16, "f32", spare=hd, pad=1, scale=1.0)


@pytest.mark.parametrize("dtype", ("f32", "f16", "bf16"))
@pytest.mark.parametrize("k_size,v_size,q_size", [(1e-3, 1e-5, 1.0), (1.0, 3000.0, 1e-4), (30.0, 1.0, 2.0)])
def test_attn_magnitudes(dtype, k_size, v_size, q_size):
    """Small and large rows keep their precision; steep scores too."""
    check_attn([300, 1000], [1, 2], 16, 2, 128, 16, dtype, k_size=k_size, v_size=v_size, q_size=q_size, seed=3)


@pytest.mark.parametrize("dtype", ("f32", "f16", "bf16"))
@pytest.mark.parametrize("hd", (64, 128, 256))
def test_attn_sixteen_heads_of_a_kv_head(hd, dtype):
    """Groups of 16: short, long and empty requests, several queries, a window with pages given back."""
    check_attn([2500, 0, 1, 47, 300], [1, 1, 1, 3, 2], 32, 2, hd, 32, dtype, seed=21)
    check_attn([900, 16, 333], [2, 1, 5], 16, 1, hd, 16, dtype, sink=20, win=130, spare=hd, pad=2, seed=22)
    check_attn([6000], [1], 16, 1, hd, 64, dtype, seed=23)
    check_attn(np.random.default_rng(24).integers(0, 60, 170).tolist(), [1] * 170, 16, 1, hd, 16, dtype, seed=24)


@pytest.mark.parametrize("hd,hq", [(64, 8), (128, 16), (256, 8)])
def test_attn_pages_that_requests_share(hd, hq):
    """Requests with a common beginning hold the same pages; one of them even twice."""
    m = fa()
    rng = np.random.default_rng(hd)
    P = 16
    pages, table, ks, vs = filled(m, rng, [160, 48], 1, hd, P)
    both = np.full((3, 13), -1)
    both[0, :10] = table[0, :10]                              # 160 rows
    both[1, :9] = np.r_[table[0, :6], table[1, :3]]           # 96 of them and the other's 48
    both[2, :13] = np.r_[table[1, :3], table[0, :10]]
    lens = [160, 140, 205]
    rows = [(ks[0], vs[0]), tuple(np.concatenate([a[:96], b]) for a, b in ((ks[0], ks[1]), (vs[0], vs[1]))),
            tuple(np.concatenate([b, a]) for a, b in ((ks[0], ks[1]), (vs[0], vs[1])))]
    q, qx = on_gpu(rng.standard_normal((3, hq, hd)), "f32")
    got = host(call_attn(m, q, ints(both), pages, ints(lens), ints([0, 1, 2, 3]), 1, P))
    for r, L in enumerate(lens):
        k, v = (x[:L] for x in rows[r])
        want, _ = ref.attend(qx[r:r + 1], L, k, v, L - 1, 0, 0, 1 / math.sqrt(hd))
        assert np.linalg.norm(got[r] - want[0]) <= 2.0 ** -17 * np.linalg.norm(want)
    both[0, 1] = both[0, 0]                                   # the same page twice in a request
    got = host(call_attn(m, q, ints(both), pages, ints(lens), ints([0, 1, 2, 3]), 1, P))
    k, v = (np.concatenate([x[:16], x[:16], x[32:]]) for x in (ks[0], vs[0]))
    want, _ = ref.attend(qx[:1], 160, k, v, 159, 0, 0, 1 / math.sqrt(hd))
    assert np.linalg.norm(got[0] - want[0]) <= 2.0 ** -17 * np.linalg.norm(want)
    assert m.get_device_error() == m.OK


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
@pytest.mark.parametrize("hd,hq", [(64, 32), (128, 8), (256, 16)])
def test_attn_infinities_and_nan_stay_in_their_rows(hd, hq, dtype):
    """A NaN or infinity in a query reaches that row alone, an infinity in a page's row the queries that attend it."""
    m = fa()
    rng = np.random.default_rng(hd)
    hkv, P, lens, nqs = 2, 16, [90, 400, 33], [2, 2, 2]
    pages, table, _, _ = filled(m, rng, lens, hkv, hd, P)
    args = ints(table), pages, ints(lens), ints(np.r_[0, np.cumsum(nqs)]), hkv, P
    q, _ = on_gpu(rng.standard_normal((6, hq, hd)), dtype)
    clean = call_attn(m, q, *args)
    for bad in (math.nan, math.inf):
        dirty = q.clone()
        dirty[2, 1, 5] = bad
        got = call_attn(m, dirty, *args)
        same = (got == clean).all(-1)
        same[2, 1] = True
        assert bool(same.all()) and bool(got[2, 1].isnan().all())
    k = torch.full((1, hkv, hd), 1.0, device="cuda")
    k[:, :, 3] = math.inf
    last = int(table[1, 399 // P]) * P + 399 % P              # the newest row of request 1: its second query's own
    v = torch.full_like(k, 1.0)
    v[:, :, 40] = math.inf
    append(m, pages, k, v, [last], P)
    got = call_attn(m, q, *args)
    keep = [0, 1, 2, 4, 5]
    assert torch.equal(got[keep], clean[keep])
    assert bool(got[3].isnan().all())
    assert m.get_device_error() == m.OK


def test_attn_refuses_more_work_than_it_counts():
    """Lengths of 2^30 rows for 65536 queries: flagged, nothing read or written."""
    m = fa()
    T, hd = 1 << 16, 64
    q = torch.zeros(T, 16, hd, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 7.0)
    table = torch.zeros(1, 1 << 22, dtype=torch.int32, device="cuda")
    call_attn(m, q, table, pool_of(m, 1, 1, hd, 256), ints([1 << 30]), ints([0, T]), 1, 256, out=out)
    assert m.get_device_error() == m.ERR_DEVICE
    assert bool((out == 7.0).all())


def test_nothing_to_do():
    """No requests, no tokens: the plan still says so, the other calls return at once."""
    m = fa()
    e = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    ring, state, cu, slots, pos = ints([1, 0]), ints([-9] * 3), ints([-9]), ints([-9] * 5), ints([-9] * 5)
    m.page_plan(e(0), e(0), ring, ints([1, 2]), e(0, 3), state, e(0), cu, slots, pos, page_rows=16)
    assert state.tolist() == [1, 2, 0] and cu.tolist() == [0] and slots.tolist() == [-1] * 5 and pos.tolist() == [0] * 5
    pages = pool_of(m, 1, 1, 64, 16)
    x = torch.zeros(0, 1, 64, device="cuda")
    m.paged_append(x, x, e(0), pages, page_rows=16)
    m.paged_attn(x, torch.zeros_like(x), e(1), e(0), e(0, 3), pages, n_kv_heads=1, page_rows=16,
                 workspace=torch.empty(m.paged_attn_workspace_bytes(64), dtype=torch.uint8, device="cuda"))
    q = torch.full((3, 8, 64), 7.0, device="cuda")            # tokens, but none of a request
    out = call_attn(m, q, e(2, 1), pages, e(2), e(3), 1, 16, out=q.clone())
    assert torch.equal(out, q)
    check_guards(("pages", pages))
    assert m.get_device_error() == m.OK


def test_attn_many_requests_of_every_length():
    rng = np.random.default_rng(8)
    lens = rng.integers(0, 200, 300).tolist()
    check_attn(lens, rng.integers(0, 3, 300).tolist(), 8, 2, 64, 16, "f32")
    lens = np.round(np.exp(rng.uniform(0, 8.5, 60))).astype(int).tolist()
    check_attn(lens, [1] * 60, 16, 2, 256, 32, "bf16")


@pytest.mark.parametrize("dtype,hd,rows", [("f32", 128, range(4000, 4700, 48)), ("bf16", 64, range(5300, 6300, 64))])
def test_attn_cuts_with_and_without_rest(dtype, hd, rows):
    """40 equal units whose lengths pass over every remainder of the cut, empty last parts of a block among them."""
    for L in rows:
        check_attn([L] * 5, [1] * 5, 8, 8, hd, 32, dtype, seed=L)


@pytest.mark.parametrize("dtype", ("f32", "f16", "bf16"))
def test_attn_cuts_of_short_units(dtype):
    """Units about as long as a warp's part, shorter and longer: most are shared by two warps."""
    for L, R, hkv in ((20, 1030, 2), (45, 700, 1), (300, 130, 2), (320, 77, 4)):
        check_attn([L] * R, [1] * R, 16 * hkv if dtype != "f32" else 4 * hkv, hkv, 128, 16, dtype, seed=L)


def test_attn_more_requests_than_threads():
    rng = np.random.default_rng(12)
    n = 3000
    lens = np.where(rng.random(n) < 0.9, rng.integers(0, 20, n), 90).tolist()
    check_attn(lens, np.where(rng.random(n) < 0.2, 0, 1).tolist(), 2, 1, 64, 16, "f16")


def test_attn_long_request():
    """A cache long enough that its rows are shared by every SM; a peak of scores at its far end."""
    check_attn([70001], [1], 8, 1, 128, 64, "f32", seed=4)
    check_attn([20000, 1], [2, 1], 16, 1, 256, 16, "bf16", seed=5)


def test_attn_pool_past_32_bits_of_bytes():
    """Pages beyond 4 GiB of the pool (and beyond 2^32 bytes of offset)."""
    m = fa()
    hkv, hd, P = 2, 256, 256
    pb = m.page_bytes(hkv, hd, P)
    n_pages = (5 << 30) // pb
    pages = torch.empty(n_pages * pb, dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(4)
    L = 300
    table = np.array([[n_pages - 1, n_pages - 7]])
    p = np.arange(L)
    slots = table[0, p // P] * P + p % P
    k, v = rng.standard_normal((2, L, hkv, hd)).astype(np.float32)
    append(m, pages, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), slots, P)
    q, qx = on_gpu(rng.standard_normal((1, 16, hd)), "f32")
    out = torch.empty_like(q)
    m.paged_attn(q, out, ints([0, 1]), ints([L]), ints(table), pages, n_kv_heads=hkv, page_rows=P,
                 workspace=torch.empty(m.paged_attn_workspace_bytes(hd), dtype=torch.uint8, device="cuda"))
    want, _ = ref.attend(qx, L, ref.decode(*ref.encode(k)), ref.decode(*ref.encode(v)), L - 1, 0, 0, 1 / 16)
    assert np.linalg.norm(host(out) - want) <= 2.0 ** -17 * np.linalg.norm(want)
    pbf = m.kv_plane_bytes(m.KV_F16, hkv, L, hd)
    kp, vp = (torch.zeros(pbf, dtype=torch.uint8, device="cuda") for _ in range(2))
    m.paged_gather(pages, ints(table), ints([L]), kp, vp, n_kv_heads=hkv, head_dim=hd, page_rows=P, max_seq=L)
    got = kp[:hkv * L * hd * 2].view(torch.float16).view(hkv, L, hd).cpu().numpy()
    assert np.array_equal(got, ref.decode(*ref.encode(k)).astype(np.float16).transpose(1, 0, 2))
    assert m.get_device_error() == m.OK


def call_attn(m, q, table, pages, lens, cu, hkv, page_rows, out=None, ws=None, **kw):
    out = torch.empty_like(q) if out is None else out
    ws = torch.empty(m.paged_attn_workspace_bytes(q.shape[2]), dtype=torch.uint8, device="cuda") if ws is None else ws
    m.paged_attn(q, out, cu, lens, table, pages, n_kv_heads=hkv, page_rows=page_rows, workspace=ws, **kw)
    return out


def test_attn_bad_device_data_is_flagged_and_skipped():
    m = fa()
    rng = np.random.default_rng(2)
    hq, hkv, hd, P = 4, 2, 64, 16
    pages, table, ks, vs = filled(m, rng, [40, 40, 40], hkv, hd, P)
    q, qx = on_gpu(rng.standard_normal((3, hq, hd)), "f32")

    def run(lens=(40, 40, 40), cu=(0, 1, 2, 3), table=table):
        out = guarded((3, hq, hd), torch.float32, fill=7.0)
        call_attn(m, q, ints(table), pages, ints(lens), ints(cu), hkv, P, out=out)
        assert m.get_device_error() == m.ERR_DEVICE
        check_guards(("out", out))
        return host(out)

    good = [ref.attend(qx[i:i + 1], 40, ks[i], vs[i], 39, 0, 0, 1 / 8)[0][0] for i in range(3)]
    ok = lambda x, i: np.linalg.norm(x - good[i]) <= 2.0 ** -17 * np.linalg.norm(good[i])  # noqa: E731
    for lens in ((40, -1, 40), (40, 49, 40), (40, 2 ** 31 - 1, 40)):
        got = run(lens=lens)
        assert np.all(got[1] == 7.0) and ok(got[0], 0) and ok(got[2], 2)
    for cu in ((0, 1, 2, 4), (0, 1, 2, 2 ** 31 - 1)):
        got = run(cu=cu)
        assert np.all(got[2] == 7.0) and ok(got[0], 0) and ok(got[1], 1)
    got = run(cu=(0, 1, 0, 3))                            # a request that ends before it begins, and one that
    assert np.all(np.isfinite(got))                       # then holds another's token: that one's row is either's
    got = run(cu=(-1, 1, 2, 3))
    assert ok(got[1], 1) and ok(got[2], 2)
    bad = table.copy()
    bad[1, 1] = 10 ** 6                                   # rows 16..31 of request 1 do not count
    got = run(table=bad)
    keep = np.r_[0:16, 32:40]
    want = ref.attend(qx[1:2], 24, ks[1][keep], vs[1][keep], 23, 0, 0, 1 / 8)[0][0]
    assert ok(got[0], 0) and ok(got[2], 2)
    assert np.linalg.norm(got[1] - want) <= 2.0 ** -17 * np.linalg.norm(want)


def test_attn_same_bits_again_and_with_other_requests_beside():
    """Two calls give the same bits; nothing depends on what the workspace holds."""
    m = fa()
    rng = np.random.default_rng(31)
    lens = [3000, 17, 900]
    pages, table, _, _ = filled(m, rng, lens, 2, 128, 32)
    q, _ = on_gpu(rng.standard_normal((3, 16, 128)), "bf16")
    ws = torch.full((m.paged_attn_workspace_bytes(128),), 0xff, dtype=torch.uint8, device="cuda")
    args = (m, q, ints(table), pages, ints(lens), ints([0, 1, 2, 3]), 2, 32)
    first = call_attn(*args, ws=ws)
    for _ in range(3):
        assert torch.equal(call_attn(*args, ws=ws), first)


def test_attn_graphs_and_streams():
    """A captured call replays with new queries, lengths and tables; two streams run two calls at once."""
    m = fa()
    rng = np.random.default_rng(13)
    hq, hkv, hd, P = 16, 2, 256, 16
    lens = [400, 90]
    pages, table, ks, vs = filled(m, rng, lens, hkv, hd, P)
    q, qx = on_gpu(rng.standard_normal((2, hq, hd)), "f32")
    t, n, cu = ints(table), ints(lens), ints([0, 1, 2])
    out, ws = torch.zeros_like(q), torch.empty(m.paged_attn_workspace_bytes(hd), dtype=torch.uint8, device="cuda")
    call_attn(m, q, t, pages, n, cu, hkv, P, out=out, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call_attn(m, q, t, pages, n, cu, hkv, P, out=out, ws=ws)
    for cut in (0, 37):
        qx = ref.round_type(rng.standard_normal(qx.shape), "f32")
        q.copy_(torch.from_numpy(qx))
        n.copy_(torch.tensor([lens[0] - cut, lens[1] - cut], dtype=torch.int32))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for r in (0, 1):
            want, _ = ref.attend(qx[r:r + 1], lens[r] - cut, ks[r], vs[r], lens[r] - cut - 1, 0, 0, 1 / 16)
            assert np.linalg.norm(host(out)[r] - want[0]) <= 2.0 ** -17 * np.linalg.norm(want)
    n.copy_(torch.tensor(lens, dtype=torch.int32))
    want = call_attn(m, q, t, pages, n, cu, hkv, P, ws=ws).clone()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros_like(q) for _ in streams]
    spaces = [torch.empty_like(ws) for _ in streams]
    for _ in range(20):
        for s, o, w in zip(streams, outs, spaces):
            call_attn(m, q, t, pages, n, cu, hkv, P, out=o, ws=w, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_a_captured_step_replays():
    """Plan, rotation, append and attention as one graph, twice over the same workspace: each replay goes on from
    the state that the one before it left, and the results are those of separate calls, bit for bit."""
    m = fa()
    R, P, max_pages, n_pages, hq, hkv, hd, T = 3, 16, 6, 14, 16, 2, 128, 24
    rope = m.rope_table(1e4 ** (-np.arange(hd // 2) / (hd // 2)))
    fresh_of = [[10, 4, 10], [1, 20, 1], [-1, 1, 1], [17, 1, 1], [1, 1, 5], [0, 0, 1]]

    def world():
        rng = np.random.default_rng(5)
        w = dict(ring=ints(rng.permutation(n_pages)), table=ints(np.full((R, max_pages), -1)),
                 lens=[ints([0] * R), ints([0] * R)], state=[ints([3, n_pages, 0]), ints([0, 0, 0])], fresh=ints([0] * R),
                 cu=ints([0] * (R + 1)), slots=ints([0] * T), pos=ints([0] * T), pages=pool_of(m, n_pages, hkv, hd, P),
                 q=torch.zeros(T, hq, hd, dtype=torch.bfloat16, device="cuda"),
                 k=torch.zeros(T, hkv, hd, dtype=torch.bfloat16, device="cuda"),
                 ws=torch.empty(m.paged_attn_workspace_bytes(hd), dtype=torch.uint8, device="cuda"),
                 out=torch.full((T, hq, hd), 7.0, dtype=torch.bfloat16, device="cuda"))
        w["v"] = torch.zeros_like(w["k"])
        return w

    def step(w, i):
        now, after = i % 2, 1 - i % 2
        m.page_plan(w["lens"][now], w["fresh"], w["ring"], w["state"][now][:2], w["table"], w["state"][after],
                    w["lens"][after], w["cu"], w["slots"], w["pos"], page_rows=P)
        m.rope(w["q"], w["k"], w["q"], w["k"], w["pos"], rope)
        m.paged_append(w["k"], w["v"], w["slots"], w["pages"], page_rows=P)
        m.paged_attn(w["q"], w["out"], w["cu"], w["lens"][after], w["table"], w["pages"], n_kv_heads=hkv, page_rows=P,
                     workspace=w["ws"])

    captured, plain = world(), world()
    step(world(), 0)                                          # the first call sets kernels up
    torch.cuda.synchronize()
    graphs = []
    for i in (0, 1):                                          # one for each side of the double buffers
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            step(captured, i)
    gen = torch.Generator("cuda").manual_seed(3)
    for i, fresh in enumerate(fresh_of):
        new = [torch.randn(T, h, hd, generator=gen, device="cuda").bfloat16() for h in (hq, hkv, hkv)]
        for w in (captured, plain):
            w["fresh"].copy_(torch.tensor(fresh, dtype=torch.int32))
            for name, x in zip("qkv", new):
                w[name].copy_(x)
        graphs[i % 2].replay()
        step(plain, i)
        torch.cuda.synchronize()
        for name in ("out", "table", "ring", "slots", "pos", "cu", "pages"):
            assert torch.equal(captured[name], plain[name]), (i, name)
        used = sum(max(f, 0) for f in fresh)
        assert bool((plain["out"][:used].float() != 7.0).any(-1).all()) and bool(torch.isfinite(plain["out"].float()).all())
    assert m.get_device_error() == m.OK


@pytest.mark.parametrize("captured", (False, True))
def test_calls_wait_for_all_that_comes_before(captured):
    """Each call's kernel may be placed before the work ahead of it is done, and has to wait for it: for copies and
    fills, for kernels of other streams, for a large kernel that still writes its input; and what follows waits too."""
    m = fa()
    R, P, hq, hkv, hd, L = 4, 16, 8, 2, 64, 40
    T, n_pages = R * L, R * 3
    rope = m.rope_table(1e4 ** (-np.arange(hd // 2) / (hd // 2)))
    gen = torch.Generator("cuda").manual_seed(11)
    src = [torch.randn(T, h, hd, generator=gen, device="cuda") for h in (hq, hkv, hkv)]
    big = torch.zeros(64 << 20, dtype=torch.float32, device="cuda")
    first = ints(np.arange(n_pages))
    pb = m.kv_plane_bytes(m.KV_F16, hkv, L, hd)
    ws = torch.empty(m.paged_attn_workspace_bytes(hd), dtype=torch.uint8, device="cuda")

    def buffers():
        return dict(q=torch.zeros_like(src[0]), k=torch.zeros_like(src[1]), v=torch.zeros_like(src[2]),
                    fresh=ints([0] * R), ring=ints([0] * n_pages), table=ints(np.full((R, 3), -1)), lens=ints([9] * R),
                    state=ints([0] * 3), cu=ints([0] * (R + 1)), slots=ints([0] * T), pos=ints([0] * T),
                    pages=pool_of(m, n_pages, hkv, hd, P), out=torch.zeros_like(src[0]),
                    planes=torch.zeros(2, R * pb, dtype=torch.uint8, device="cuda"), lens0=ints([0] * R),
                    state0=ints([0, n_pages]), sum=torch.zeros(4, dtype=torch.float64, device="cuda"))

    def work(b, wait):
        """wait: the host waits after every step, so that nothing can overlap."""
        def next_():
            if wait:
                torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):                     # q and v come from another stream, late
            big.add_(1.0)
            b["q"].copy_(src[0]); b["v"].copy_(src[2])
        b["fresh"].fill_(L); next_()
        b["ring"].copy_(first); next_()
        m.page_plan(b["lens0"], b["fresh"], b["ring"], b["state0"], b["table"], b["state"], b["lens"], b["cu"],
                    b["slots"], b["pos"], page_rows=P); next_()
        b["k"].copy_(src[1])
        torch.cuda.current_stream().wait_stream(side); next_()
        m.rope(b["q"], b["k"], b["q"], b["k"], b["pos"], rope); next_()
        m.paged_append(b["k"], b["v"], b["slots"], b["pages"], page_rows=P); next_()
        m.paged_gather(b["pages"], b["table"], b["lens"], *b["planes"], n_kv_heads=hkv, head_dim=hd, page_rows=P,
                       max_seq=L); next_()
        m.paged_attn(b["q"], b["out"], b["cu"], b["lens"], b["table"], b["pages"], n_kv_heads=hkv, page_rows=P,
                     workspace=ws); next_()
        b["sum"][0] = b["out"].double().sum()
        b["q"].zero_(); next_()                           # the queries may be overwritten after the call
        m.rope(b["out"], None, b["q"], None, b["pos"], rope, inverse=True); next_()
        b["sum"][1] = b["q"].double().sum()
        big.mul_(0.5)

    want, got = buffers(), buffers()
    work(want, True)
    torch.cuda.synchronize()
    if captured:
        work(buffers(), False)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            work(got, False)
        for _ in range(3):
            graph.replay()
    else:
        work(got, False)
    torch.cuda.synchronize()
    for name in want:
        assert torch.equal(got[name], want[name]), name
    assert bool(torch.isfinite(want["sum"][:2]).all()) and float(want["sum"][0]) != 0
    assert m.get_device_error() == m.OK


def test_paged_refuses_shapes_and_types():
    m = fa()
    P, hkv, hd = 16, 2, 64
    pages = m.alloc_pages(4, hkv, hd, P)
    x = torch.zeros(3, hkv, hd, device="cuda")
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    slots, table, lens, cu = i32(3), i32(2, 2), i32(2), i32(3)
    planes = torch.zeros(2 * m.kv_plane_bytes(m.KV_F16, hkv, 32, hd), dtype=torch.uint8, device="cuda")
    ws = torch.zeros(m.paged_attn_workspace_bytes(hd), dtype=torch.uint8, device="cuda")
    q = torch.zeros(3, 4, hd, device="cuda")
    bad_calls = [
        lambda: m.paged_append(x, x[:2], slots, pages, page_rows=P),
        lambda: m.paged_append(x, x.half(), slots, pages, page_rows=P),
        lambda: m.paged_append(x, x, slots[:2], pages, page_rows=P),
        lambda: m.paged_append(x, x, slots, pages[:-1], page_rows=P),
        lambda: m.paged_append(x, x, slots, pages, page_rows=17),
        lambda: m.paged_append(x.double(), x.double(), slots, pages, page_rows=P),
        lambda: m.paged_append(x.transpose(1, 2), x.transpose(1, 2), slots, pages, page_rows=P),
        lambda: m.paged_append(x[:1].expand(3, hkv, hd), x, slots, pages, page_rows=P),
        lambda: m.paged_append(x.cpu(), x, slots, pages, page_rows=P),
        lambda: m.paged_gather(pages, table, i32(3), planes, planes, n_kv_heads=hkv, head_dim=hd, page_rows=P,
                               max_seq=32),
        lambda: m.paged_gather(pages, table, lens, planes[:-256], planes, n_kv_heads=hkv, head_dim=hd, page_rows=P,
                               max_seq=32),
        lambda: m.paged_gather(pages, table.long(), lens, planes, planes, n_kv_heads=hkv, head_dim=hd, page_rows=P,
                               max_seq=32),
        lambda: m.paged_attn(q, q[:2], cu, lens, table, pages, n_kv_heads=hkv, page_rows=P, workspace=ws),
        lambda: m.paged_attn(q, q.half(), cu, lens, table, pages, n_kv_heads=hkv, page_rows=P, workspace=ws),
        lambda: m.paged_attn(q, q, cu[:2], lens, table, pages, n_kv_heads=hkv, page_rows=P, workspace=ws),
        lambda: m.paged_attn(q, q, cu, lens, table[0], pages, n_kv_heads=hkv, page_rows=P, workspace=ws),
        lambda: m.paged_attn(q, q, cu, lens, table, pages, n_kv_heads=hkv, page_rows=P, workspace=ws,
                             lse=torch.zeros(3, 4, device="cuda")),
        lambda: m.paged_attn(q, q, cu, lens, table, pages.cpu(), n_kv_heads=hkv, page_rows=P, workspace=ws),
    ]
    for i, bad in enumerate(bad_calls):
        with pytest.raises(ValueError):
            bad()
            pytest.fail(f"call {i} was taken")
    for kw in (dict(n_kv_heads=hkv, workspace=ws[:64]), dict(n_kv_heads=hkv, workspace=ws, sink=-1),
               dict(n_kv_heads=hkv, workspace=ws, scale=-0.5)):
        with pytest.raises(m.FAError):
            m.paged_attn(q, q, cu, lens, table, pages, page_rows=P, **kw)
    with pytest.raises(m.FAError):  # rows that 16-byte loads cannot read
        y = torch.zeros(3, hkv * hd + 1, device="cuda")[:, :hkv * hd].unflatten(1, (hkv, hd))
        m.paged_append(y, y, slots, pages, page_rows=P)


# ------------------------------------------------- a run of them together

def test_serving_steps(oracle_mod):
    """Five steps of a small server: prompts, a chunk, decodes, a finished request whose pages go to the next.
    Every step plans, rotates, appends and attends; the prompts also go through fp16 planes and fa_prefill_chunk."""
    m = fa()
    rng = np.random.default_rng(77)
    R, P, max_pages, n_pages, hq, hkv, hd = 4, 16, 12, 20, 8, 2, 64
    freq = 1e4 ** (-np.arange(16) / 16)
    axis = ref.axes_of(16, [16], False)
    table_rope = m.rope_table(freq)
    pages = pool_of(m, n_pages, hkv, hd, P)
    ring, table = ints(rng.permutation(n_pages)), ints(np.full((R, max_pages), -1))
    lens, state = [ints([0] * R), ints([0] * R)], [ints([5, n_pages, 0]), ints([0, 0, 0])]
    cache = [(np.zeros((0, hkv, hd)), np.zeros((0, hkv, hd))) for _ in range(R)]
    ws = torch.empty(m.paged_attn_workspace_bytes(hd), dtype=torch.uint8, device="cuda")
    max_tokens = 170
    steps = [[70, 33, 0, 5], [1, 1, 90, 1], [1, -1, 1, 1], [1, 120, 1, 2], [1, 1, -1, 1]]
    for i, fresh in enumerate(steps):
        now, after = i % 2, 1 - i % 2
        cu, slots, pos = ints([0] * (R + 1)), ints([0] * max_tokens), ints([0] * max_tokens)
        m.page_plan(lens[now], ints(fresh), ring, state[now][:2], table, state[after], lens[after], cu, slots, pos,
                    page_rows=P)
        T = sum(max(f, 0) for f in fresh)
        # the batch is padded to max_tokens, as a captured step's is
        qkv = torch.from_numpy(rng.standard_normal((max_tokens, hq + 2 * hkv, hd)).astype(np.float32)).cuda()
        q, k, v = qkv.split([hq, hkv, hkv], 1)
        qx, kx, vx = (host(x)[:T] for x in (q, k, v))
        positions = pos.cpu().numpy()[None, :T]
        m.rope(q, k, q, k, pos, table_rope)
        m.paged_append(k, v, slots, pages, page_rows=P)
        out, lse = torch.full((max_tokens, hq, hd), 7.0, device="cuda"), torch.empty(hq, max_tokens, device="cuda")
        m.paged_attn(q, out, cu, lens[after], table, pages, n_kv_heads=hkv, page_rows=P, lse=lse, workspace=ws)
        assert m.get_device_error() == m.OK
        assert bool((out[T:] == 7.0).all())
        qx = ref.rope(qx, positions, freq, axis, False, False)
        kr = host(k)[:T]  # as rotated in fp32: the codes follow it bit for bit
        assert np.allclose(kr, ref.rope(kx, positions, freq, axis, False, False), atol=2e-6, rtol=0)
        t = 0
        for r, f in enumerate(fresh):
            if f < 0:
                cache[r] = (np.zeros((0, hkv, hd)), np.zeros((0, hkv, hd)))
                continue
            new = [ref.decode(*ref.encode(x[t:t + f].astype(np.float32))) for x in (kr, vx)]
            cache[r] = tuple(np.concatenate([a, b]) for a, b in zip(cache[r], new))
            L = len(cache[r][0])
            assert int(lens[after][r]) == L
            want, _ = ref.attend(qx[t:t + f], L, *cache[r], L - f, 0, 0, 1 / 8)
            got = host(out)[t:t + f]
            if f:
                # 2^-17 of the kernel, and rope's 2e-6 on q: scores of |q| |k| / 8 <= 2e-6 * 64 * 3 / 8
                assert np.linalg.norm(got - want) <= (2.0 ** -17 + 1e-4) * np.linalg.norm(want)
            if f > 1:  # the chunk by way of planes
                max_seq = L + 2
                pb = m.kv_plane_bytes(m.KV_F16, hkv, max_seq, hd)
                kp, vp = (torch.zeros(pb, dtype=torch.uint8, device="cuda") for _ in range(2))
                m.paged_gather(pages, table[r:r + 1], lens[after][r:r + 1], kp, vp, n_kv_heads=hkv, head_dim=hd,
                               page_rows=P, max_seq=max_seq)
                o = torch.empty(f, hq, hd, device="cuda")
                m.prefill_chunk(q[t:t + f].contiguous(), kp, vp, o, L - f, f, hq, hkv, hd, 0, 0, m.KV_F16,
                                max_seq=max_seq, workspace=torch.empty(
                                    m.prefill_chunk_workspace_bytes(L - f, f, hq, hkv, hd), dtype=torch.uint8,
                                    device="cuda"))
                assert np.abs(host(o) - want).max() <= 5e-3  # the prefill's own tolerance (fp16 operands)
                assert m.get_device_error() == m.OK
            t += f


# ------------------------------- sums and references whatever the values are

@pytest.mark.parametrize("dtype", ("f32", "f16", "bf16"))
@pytest.mark.parametrize("hd,hq", [(64, 16), (128, 8), (256, 16)])
def test_attn_sums_do_not_depend_on_the_size_of_v(hd, hq, dtype):
    """V next to the smallest and the largest fp32 numbers: the log-sum-exp and the weights know nothing of it.
    (1e-36: outputs are averages, still above 1.2e-38, where a half step would no longer be relative.)"""
    for lens, v_size in (([8192], 1e-33), ([600, 40], 1e-34), ([300], 1e-36), ([700], 1e30), ([300, 7], 3e37)):
        if dtype == "f16" and v_size > 1:
            continue  # not binary16 numbers
        check_attn(lens, [1] * len(lens), hq, 1, hd, 16, dtype, v_size=v_size, seed=41)


@pytest.mark.parametrize("dtype", ("f32", "f16", "bf16"))
@pytest.mark.parametrize("hd,hq", [(64, 16), (128, 4), (256, 8)])
def test_attn_rows_of_v_of_all_sizes(hd, hq, dtype):
    """Rows of 1e-36 before, behind and among ordinary ones."""
    rng = np.random.default_rng(3)
    L = 1024
    small_first = np.where(np.arange(L) < 16, 1e-36, 1.0)
    some = 10.0 ** rng.uniform(-30, 3, L)
    for sizes in (small_first, small_first[::-1], np.where(np.arange(L) % 64 < 63, 1e-36, 1.0), some):
        check_attn([L], [2], hq, 1, hd, 16, dtype, v_size=sizes[:, None, None], seed=43)


def attend_filled(m, rng, k, v, hq, hkv, hd, page_rows, dtype, n_q, q=None):
    """One request of rows k, v [L][hkv][hd] and n_q queries: (out [n_q][hq][hd], lse [hq][n_q], q as rounded)."""
    L = len(k)
    used = -(-L // page_rows)
    pages = pool_of(m, used + 1, hkv, hd, page_rows)
    table = rng.permutation(used + 1)[:used][None]
    p = np.arange(L)
    append(m, pages, torch.from_numpy(k.astype(np.float32)).cuda(), torch.from_numpy(v.astype(np.float32)).cuda(),
           table[0, p // page_rows] * page_rows + p % page_rows, page_rows)
    q, qx = on_gpu(rng.standard_normal((n_q, hq, hd)) if q is None else q, dtype)
    lse = guarded((hq, n_q), torch.float32, fill=7.0)
    out = call_attn(m, q, ints(table), pages, ints([L]), ints([0, n_q]), hkv, page_rows, lse=lse)
    assert m.get_device_error() == m.OK
    check_guards(("lse", lse))
    return host(out), host(lse), qx


@pytest.mark.parametrize("dtype", ("f32", "f16", "bf16"))
@pytest.mark.parametrize("hd,hq", [(64, 16), (128, 4), (256, 8)])
def test_attn_rows_of_zeros_do_not_hide_the_others(hd, hq, dtype):
    """A null token whose V is zero and whose score is far above all others: what the others give keeps its bits."""
    m = fa()
    rng = np.random.default_rng(hd)
    for L, bits, size in ((8192, 20, 1e-2), (8192, 20, 1e-3), (2000, 11, 1e-5), (100, 3, 1e-20), (40, 6, 0.0)):
        k = 0.02 * rng.standard_normal((L, 1, hd))
        k[0] = bits * math.log(2) / math.sqrt(hd)             # q . k0 / sqrt(hd) is `bits` powers of two above the rest
        v = size * (1 + 0.3 * rng.standard_normal((L, 1, hd)))
        v[[0, L // 2, L - 1]] = 0
        got, lse, qx = attend_filled(m, rng, k, v, hq, 1, hd, 32, dtype, 2, q=1 + 0.1 * rng.standard_normal((2, hq, hd)))
        kx, vx = (ref.decode(*ref.encode(x.astype(np.float32))) for x in (k, v))
        want, wl = ref.attend(qx, L, kx, vx, L - 2, 0, 0, 1 / math.sqrt(hd))
        # The largest score has an error of at most 16 half steps at its size (the sums of 8 blocks, their products in
        # the tensor core, the scale and the exponent): 16 * bits * 2^-24 of its weight. The 16-bit types' scores have
        # their codes' offset in the sums besides, 9 * 2^-23 * 23 / 7 of the score; then their output's rounding.
        tol = {"f32": bits * 2.0 ** -20 + 2.0 ** -17, "f16": bits * 2.0 ** -18 + 2.0 ** -10,
               "bf16": bits * 2.0 ** -18 + 2.0 ** -8}[dtype]
        floor = 2.0 ** -25 * math.sqrt(want.size) if dtype == "f16" else 0.0
        assert np.linalg.norm(got - want) <= tol * np.linalg.norm(want) + floor, (L, bits, size)
        assert np.all(np.abs(lse - wl) <= (bits + 1) * 2.0 ** -18 + np.abs(wl) * 2.0 ** -22)


@pytest.mark.parametrize("dtype", ("f32", "f16", "bf16"))
@pytest.mark.parametrize("hd,hq", [(64, 32), (128, 8), (256, 16)])
def test_attn_an_infinity_in_v_reaches_its_block_alone(hd, hq, dtype):
    """V with an infinity in one block of a row: that block is NaN for the queries that attend the row, also where its
    weight is nothing; the other blocks (0 in such a row) and the log-sum-exp are what the definition gives."""
    m = fa()
    hkv, L, n_q = 2, 300, 3
    for row, low in ((150, False), (L - 1, False), (L - 2, True), (20, True)):
        rng = np.random.default_rng(hd + row)
        k, v = rng.standard_normal((2, L, hkv, hd))
        q = 1 + 0.5 * rng.standard_normal((n_q, hq, hd))
        if low:
            k[row] = -60                                      # a score of about -60 sqrt(hd): its weight is 0 in fp32
        v[row, :, 40] = math.inf
        got, lse, qx = attend_filled(m, rng, k, v, hq, hkv, hd, 16, dtype, n_q, q=q)
        v[row] = 0
        kx, vx = (ref.decode(*ref.encode(x.astype(np.float32))) for x in (k, v))
        want, wl = ref.attend(qx, L, kx, vx, L - n_q, 0, 0, 1 / math.sqrt(hd))
        tol, ltol = attn_bounds(qx, kx, vx, dtype, 1 / math.sqrt(hd))
        tol = tol + ref.HALF_STEP[dtype] * (np.abs(want) + tol) + (2.0 ** -25 if dtype == "f16" else 0.0)
        sees = np.arange(n_q) + L - n_q >= row
        bad = np.zeros(got.shape, bool)
        bad[sees, :, 32:64] = True
        assert np.array_equal(np.isnan(got), bad), (row, low)
        assert np.all(np.abs(got - want)[~bad] <= tol[~bad]), (row, low)
        assert np.all(np.abs(lse - wl) <= ltol.T + np.abs(wl) * 2.0 ** -22), (row, low)


@pytest.mark.parametrize("tokens", range(0, 75))
def test_plan_with_too_few_tokens_gives_the_others_all(tokens):
    """max_tokens below the step's tokens: a request that it cuts gets no page, no slot and no length, those before it
    all of theirs, and lengths, offsets and the ring say the same. A step after that goes on from there."""
    m = fa()
    rng = np.random.default_rng(1)
    cached, fresh = np.array([0, 16, 3, 31, 7, 7, 0, 60]), np.array([20, 1, 0, 2, -1, 9, 33, 5])
    used = -(-cached // 16)
    order, table, at = rng.permutation(40), np.full((8, 6), -1), 0
    for r in range(8):
        table[r, :used[r]] = order[at:at + used[r]]
        at += used[r]
    ring = np.full(40, -7)
    ring[(35 + np.arange(40 - at)) % 40] = order[at:]
    step = (cached, fresh, ring, [35, 40 - at], table)
    ends = np.cumsum(np.maximum(fresh, 0))
    gone = (fresh > 0) & (ends > tokens)
    _, got = run_plan(*step, 16, tokens)
    assert m.get_device_error() == (m.ERR_DEVICE if gone.any() else m.OK)
    want = ref.plan(cached, np.where(gone, 0, fresh), *step[2:], 16, max(tokens, ends[-1]))
    for name in ("ring", "table", "lens"):
        assert got[name] == [list(map(int, x)) if name == "table" else int(x) for x in want[name]], name
    needs = -(-(cached + np.maximum(fresh, 0)) // 16) - used
    assert got["state"] == [int(x) for x in want["state"][:2]] + [int(needs[gone].sum())]
    assert got["cu"] == [0] + np.minimum(ends, tokens).tolist()
    kept = int(np.maximum(fresh[~gone], 0).sum())
    assert got["slots"] == ([int(x) for x in want["slots"][:kept]] + [-1] * tokens)[:tokens]
    pos = np.concatenate([np.arange(c, c + max(f, 0)) for c, f in zip(cached, fresh)])
    assert got["positions"] == np.r_[pos, np.zeros(tokens, int)][:tokens].astype(int).tolist()
    # the rest in a step of its own: every page is some request's or free, once
    step = (np.array(got["lens"]), np.where(gone, fresh, 0), got["ring"], got["state"][:2], np.array(got["table"]))
    _, then = run_plan(*step, 16, 80)
    want = ref.plan(*step, 16, 80)
    for name in want:
        assert then[name] == [list(map(int, x)) if name == "table" else int(x) for x in want[name]], name
    assert m.get_device_error() == m.OK
    held = [p for r, n in enumerate(then["lens"]) for p in then["table"][r][:-(-n // 16)]]
    head, count = then["state"][:2]
    assert sorted(held + [then["ring"][(head + i) % 40] for i in range(count)]) == list(range(40))


@pytest.mark.parametrize("dtype,adjacent", [("f32", False), ("bf16", True)])
def test_rope_table_of_more_axes_than_positions(dtype, adjacent):
    """A table for three axes with positions of two, and one whose entries name no axis at all: flagged, and the
    pairs that have no positions are left as they are."""
    m = fa()
    rng = np.random.default_rng(4)
    T, H, hd, half = 9, 3, 64, 32
    freq = 1e4 ** (-np.arange(half) / half)
    sections = [12, 10, 10]
    axis = ref.axes_of(half, sections, False)
    x, exact = on_gpu(rng.standard_normal((T, H, hd)), dtype)
    pos = rng.integers(0, 100, (3, T))
    table = m.rope_table(freq, sections)
    want = torch.empty_like(x)
    m.rope(x, None, want, None, ints(pos), table, adjacent=adjacent)
    assert m.get_device_error() == m.OK
    i = np.arange(half)
    lo, hi = (2 * i, 2 * i + 1) if adjacent else (i, i + half)
    for entries, value in ((axis == 2, 2), (i % 5 == 0, -1), (i == 7, 2 ** 31 - 1), (i >= 30, -2 ** 31)):
        bad = table.clone()
        bad[torch.from_numpy(entries).cuda(), 2] = value
        n_axes = 2 if value == 2 else 3
        out = guarded((T, H, hd), DT[dtype], fill=float("nan"))
        m.rope(x, None, out, None, ints(pos[:n_axes]), bad, adjacent=adjacent)
        assert m.get_device_error() == m.ERR_DEVICE
        check_guards(("out", out))
        still = np.r_[lo[entries], hi[entries]]
        assert np.array_equal(host(out)[..., still], exact[..., still])
        rest = np.setdiff1d(np.arange(hd), still)
        assert np.array_equal(host(out)[..., rest], host(want)[..., rest])


@pytest.mark.parametrize("c", (1, 3, 4, 5, 6, 7, 8, 9, 13))
def test_attn_parts_of_a_few_groups(c):
    """About c measures of the cut (a unit's groups, and 3 for its start) for each block: with 5, 6 and 9 a warp's
    part is as long as a unit's start, and some hold no group at all."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for groups in (1, 2, 5, 40):
        for more in (-1, 0, 1):
            n = max(1, c * sms // (groups + 3) + more)
            check_attn([16 * groups - 3] * n, [1] * n, 4, 1, 64, 16, "f32", seed=groups)


def test_rope_refuses_positions_and_tables_without_dims():
    m = fa()
    table = m.rope_table([1.0] * 16)
    x = torch.zeros(4, 2, 32, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    for p, t in ((pos[0], table), (pos[None, None], table), (pos, table[0, 0]), (pos, table[0])):
        with pytest.raises(ValueError):
            m.rope(x, None, x, None, p, t)


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
@pytest.mark.parametrize("hd,hq", [(64, 16), (256, 4)])
def test_attn_scores_far_below_zero(hd, hq, dtype):
    """Scores of about -1e31, and of 1e31: rows are attended, and the log-sum-exp is of the scores' size."""
    m = fa()
    rng = np.random.default_rng(hd)
    for L in (5, 700):
        for sign in (-1.0, 1.0):
            k = np.full((L, 1, hd), sign * 2.0 ** 50)
            v = rng.standard_normal((L, 1, hd))
            got, lse, qx = attend_filled(m, rng, k, v, hq, 1, hd, 16, dtype, 2, q=np.full((2, hq, hd), 2.0 ** 50))
            kx, vx = (ref.decode(*ref.encode(x.astype(np.float32))) for x in (k, v))
            _, wl = ref.attend(qx, L, kx, vx, L - 2, 0, 0, 1 / math.sqrt(hd))
            # A score of this size has an error of up to half an fp32 step, 2^-24 of 2^103: a weight, 2 to the power of
            # it, may be any, V's exponent next to the score included. What is left of the definition: outputs are
            # averages of the seen rows, to the type's rounding (and fp32 sums' 2^-17), and lse has its score's rounding.
            slack = {"f32": 2.0 ** -17, "bf16": 2.0 ** -7}[dtype] * np.abs(vx).max()
            assert np.all(got <= vx.max(0) + slack) and np.all(got >= vx.min(0) - slack)
            assert np.all(np.abs(got).max(-1) >= slack)
            assert np.all(np.abs(lse - wl) <= 2.0 ** -19 * np.abs(wl))
