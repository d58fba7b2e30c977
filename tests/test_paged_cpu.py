"""Paged serving without a GPU: what fa_page_plan, fa_rope, fa_paged_append,
fa_paged_gather and fa_paged_attn refuse before any launch, the rotation table
in closed form, and pins of the reference that the GPU tests compare with."""
import ctypes
import math

import numpy as np
import pytest

import paged_ref as ref


@pytest.fixture(scope="module")
def fa():
    from causal_gqa_flash_attn_gb300 import build
    build.build()
    import causal_gqa_flash_attn_gb300 as fa
    fa.lib()
    return fa


def caller(fn, names, **base):
    """A call by keyword whose other arguments are valid (pointers are 16: aligned, never read)."""
    def call(**kw):
        a = {**base, **kw}
        return fn(*[a[n] for n in names])
    return call


def test_page_bytes(fa):
    for hd in (64, 128, 256):
        assert fa.page_bytes(1, hd, 16) == 18 * hd + 64
        assert fa.page_bytes(3, hd, 256) == 3 * 16 * (18 * hd + 64)
    for bad in ((0, 64, 16), (2, 96, 16), (2, 100, 16), (2, 64, 8), (2, 64, 48), (2, 64, 512)):
        assert fa.page_bytes(*bad) == 0


def test_plan_refusals(fa):
    names = ("cached fresh n ring n_pages state state_out table max_pages rows lens cu slots pos "
             "max_tokens stream").split()
    call = caller(fa.lib().fa_page_plan, names, cached=16, fresh=16, n=4, ring=16, n_pages=10,
                  state=16, state_out=32, table=16, max_pages=4, rows=16, lens=32, cu=16, slots=16,
                  pos=16, max_tokens=4, stream=None)
    for bad in (dict(n=-1), dict(max_tokens=-1), dict(rows=20), dict(rows=8), dict(n_pages=0),
                dict(max_pages=0), dict(n_pages=1 << 27), dict(max_pages=1 << 27), dict(ring=None),
                dict(state=None), dict(state_out=None), dict(cu=None), dict(cached=None),
                dict(fresh=None), dict(table=None), dict(lens=None), dict(slots=None),
                dict(pos=None), dict(cached=18), dict(pos=18), dict(state_out=16), dict(lens=16)):
        assert call(**bad) == fa.ERR_INVALID, bad
    assert call(n=16385) == fa.ERR_UNSUPPORTED
    assert call(max_tokens=(1 << 30) + 1) == fa.ERR_UNSUPPORTED


def test_rope_refusals(fa):
    names = ("q q_out k k_out type n hq hkv hd rd qs qos ks kos pos pos_stride axes table adjacent "
             "inverse stream").split()
    call = caller(fa.lib().fa_rope, names, q=16, q_out=32, k=16, k_out=32, type=0, n=4, hq=4, hkv=2,
                  hd=64, rd=64, qs=256, qos=256, ks=128, kos=128, pos=16, pos_stride=4, axes=1,
                  table=16, adjacent=0, inverse=0, stream=None)
    for bad in (dict(type=3), dict(n=-1), dict(hd=1), dict(rd=0), dict(rd=7), dict(rd=66),
                dict(axes=0), dict(axes=9), dict(q=None), dict(q_out=None), dict(k=None),
                dict(k_out=None), dict(q=18), dict(qs=255), dict(kos=127), dict(qs=1 << 60),
                dict(q_out=16, qos=512), dict(pos=None), dict(pos=18), dict(pos_stride=3),
                dict(table=None), dict(table=24), dict(hq=-1)):
        assert call(**bad) == fa.ERR_INVALID, bad
    assert call(n=0) == fa.OK
    assert call(hq=0, hkv=0) == fa.OK


def test_rope_table_closed_form_and_refusals(fa):
    half = 24
    freq = 1e4 ** (-np.arange(half) / half)
    for sections, interleaved in (([24], False), ([8, 10, 6], False), ([12, 6, 6], True), ([12, 12], True)):
        t = fa.rope_table(freq, sections, interleaved=interleaved, device="cpu").numpy().view(np.uint32)
        got = (t[:, 0].astype(np.float64) + t[:, 1].astype(np.float64) * 2.0 ** 32) / 2.0 ** 64
        # inv_freq / (2 pi) in double: half a step for the division, one for 2 pi's own rounding;
        # the entry is cut to whole steps of 2^-64, and `got` is rounded from 64 bits to 53
        assert np.all(np.abs(got - freq / (2 * math.pi)) <= freq * 2.0 ** -53 + 2.0 ** -64)
        assert t[:, 2].tolist() == ref.axes_of(half, sections, interleaved).tolist()
        assert not t[:, 3].any()
    for bad in (([23], False), ([-1, 25], False), ([20, 2, 2, 0, 0, 0, 0, 0, 0], False), ([8, 8, 9], False),
                ([2, 11, 11], True)):
        with pytest.raises(fa.FAError):
            fa.rope_table(freq, bad[0], interleaved=bad[1], device="cpu")
    for bad in (float("nan"), float("inf"), -1.0):
        with pytest.raises(fa.FAError):
            fa.rope_table([1.0, bad], device="cpu")
    one = (ctypes.c_int * 1)(2)
    assert fa.lib().fa_rope_table(None, None, 2, one, 1, 0) == fa.ERR_INVALID


def test_append_refusals(fa):
    names = "k v type ks vs slots n pages n_pages hkv hd rows stream".split()
    call = caller(fa.lib().fa_paged_append, names, k=16, v=16, type=2, ks=128, vs=128, slots=16, n=4,
                  pages=16, n_pages=4, hkv=2, hd=64, rows=16, stream=None)
    for bad in (dict(type=-1), dict(n=-1), dict(n_pages=0), dict(n_pages=1 << 27), dict(k=None),
                dict(v=None), dict(slots=None), dict(pages=None), dict(k=8), dict(slots=18),
                dict(pages=24), dict(ks=127), dict(ks=132), dict(vs=100), dict(hkv=0), dict(hd=48),
                dict(rows=24)):
        assert call(**bad) == fa.ERR_INVALID, bad
    assert call(hd=96) == fa.ERR_UNSUPPORTED
    assert call(n=(1 << 30) + 1) == fa.ERR_UNSUPPORTED
    assert call(hkv=65536, ks=1 << 22, vs=1 << 22) == fa.ERR_UNSUPPORTED
    assert call(n=0) == fa.OK


def test_gather_refusals(fa):
    names = "pages n_pages table max_pages lens n hkv hd rows kp vp max_seq stream".split()
    call = caller(fa.lib().fa_paged_gather, names, pages=16, n_pages=4, table=16, max_pages=2, lens=16,
                  n=2, hkv=2, hd=64, rows=16, kp=16, vp=16, max_seq=32, stream=None)
    for bad in (dict(n=-1), dict(n_pages=0), dict(max_pages=0), dict(max_seq=0), dict(pages=None),
                dict(table=None), dict(lens=None), dict(kp=None), dict(vp=None), dict(pages=8),
                dict(table=18), dict(kp=24), dict(hkv=0), dict(rows=0)):
        assert call(**bad) == fa.ERR_INVALID, bad
    assert call(hd=96) == fa.ERR_UNSUPPORTED
    assert call(n=65536) == fa.ERR_UNSUPPORTED
    assert call(max_seq=(1 << 30) + 1) == fa.ERR_UNSUPPORTED
    assert call(n=0) == fa.OK


def test_attn_refusals(fa):
    names = ("q out lse type qs os cu lens table max_pages pages n_pages rows n_reqs n_tokens hq hkv hd "
             "sink win scale ws wsb stream").split()
    call = caller(fa.lib().fa_paged_attn, names, q=16, out=16, lse=None, type=0, qs=512, os=512, cu=16,
                  lens=16, table=16, max_pages=2, pages=16, n_pages=4, rows=16, n_reqs=2, n_tokens=2,
                  hq=8, hkv=2, hd=64, sink=0, win=0, scale=0.0, ws=16, wsb=1 << 30, stream=None)
    for bad in (dict(type=3), dict(hq=0), dict(hq=7), dict(hkv=0), dict(hd=72), dict(n_reqs=-1),
                dict(n_tokens=-1), dict(sink=-1), dict(n_pages=0), dict(max_pages=0), dict(rows=12),
                dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(q=None),
                dict(out=None), dict(cu=None), dict(lens=None), dict(table=None), dict(pages=None),
                dict(ws=None), dict(q=8), dict(out=8), dict(lse=18), dict(cu=18), dict(pages=8),
                dict(ws=8), dict(qs=511), dict(qs=514), dict(os=100)):
        assert call(**bad) == fa.ERR_INVALID, bad
    for bad in (dict(hd=96), dict(hq=24), dict(hq=64), dict(n_reqs=65537)):
        assert call(**bad) == fa.ERR_UNSUPPORTED, bad
    assert call(wsb=fa.paged_attn_workspace_bytes(64) - 1) == fa.ERR_WORKSPACE
    assert call(q=32, out=32) == fa.ERR_INVALID           # in place
    assert call(hq=1 << 17, hkv=1 << 16, qs=1 << 23, os=1 << 23, n_tokens=1) == fa.ERR_UNSUPPORTED
    assert call(n_reqs=0) == fa.OK
    assert call(n_tokens=0) == fa.OK
    for hd in (64, 128, 256):
        assert 0 < fa.paged_attn_workspace_bytes(hd) <= 64 << 20
    assert fa.paged_attn_workspace_bytes(96) == 0


# ------------------------------------------------------ pins of the reference

@pytest.mark.parametrize("hd", (64, 128, 256))
def test_places_cover_a_group_once(hd):
    """Every 4-bit code, scale and factor of a group has its own place and the group has no gap."""
    seen = np.zeros(group := ref.group_bytes(hd), np.int64)
    for v in (0, 1):
        base = v * group // 2
        for r in range(16):
            for e in range(hd):
                byte, shift = ref.code_place(hd, r, e, v)
                seen[base + byte] += 1 << shift
            for b in range(hd // 32):
                o = base + ref.scale_place(hd, r, b, v)
                seen[o:o + 2] += 17
            seen[base + 9 * hd + 2 * r:base + 9 * hd + 2 * r + 2] += 17
    assert np.all(seen == 17)  # one visit of each half byte


def test_rows_hold_the_values_of_q4_planes(oracle_mod):
    """In binary16's normal range a page row stands for exactly what a Q4_0 plane row stands for."""
    rng = np.random.default_rng(5)
    x = rng.standard_normal((40, 256)).astype(np.float32) * np.float32(3)
    x[3, 32:64] = 0
    want = oracle_mod.q4_decode(oracle_mod.q4_encode(x), 256)
    assert np.array_equal(ref.decode(*ref.encode(x)), want)
    # and outside it, a relative error of a step at most: half a code (or a whole one at -amax), and the
    # scale's rounding on codes up to 8
    for size in (1e-6, 1e6, 1e-20, 1e20):
        y = x * np.float32(size)
        d = np.abs(y.astype(np.float64).reshape(40, 8, 32)).max(-1, keepdims=True) / 8
        off = np.abs(ref.decode(*ref.encode(y)).reshape(40, 8, 32) - y.reshape(40, 8, 32))
        assert np.all(off <= d * (1 + 8 * 2.0 ** -11))


def test_reference_attention_closed_forms():
    rng = np.random.default_rng(6)
    k, v = rng.standard_normal((2, 9, 2, 64))
    q = rng.standard_normal((3, 4, 64))
    out, lse = ref.attend(q, 9, np.zeros_like(k), v, 6, 0, 0, 1.0)  # equal scores: the mean of what is seen
    for i in range(3):
        assert np.allclose(out[i], np.repeat(v[:7 + i].mean(0), 2, 0), atol=1e-14)
        assert np.allclose(lse[:, i], math.log(7 + i))
    out, lse = ref.attend(q, 2, k, v, -1, 0, 0, 1.0)                # a query before the first row
    assert not out[0].any() and np.all(lse[:, 0] == -math.inf)
    assert np.allclose(out[1], np.repeat(v[0], 2, 0))
    out, _ = ref.attend(q, 9, k, v, 6, 0, 1, 1.0)                   # a window of one: its own row
    assert np.allclose(out[2], np.repeat(v[8], 2, 0))


def test_reference_plan_by_hand():
    got = ref.plan([15, 32, 5, 0], [3, 1, -1, 16], [9, 8, 7, 6, 5, 4], [4, 4], [[0, -1, -1], [1, 2, -1], [3, -1, -1],
                   [-1, -1, -1]], 16, 22)
    assert got["table"] == [[0, 5, -1], [1, 2, 4], [3, -1, -1], [9, -1, -1]]
    assert got["lens"] == [18, 33, 0, 16] and got["cu"] == [0, 3, 4, 4, 20]
    assert got["slots"][:5] == [15, 80, 81, 64, 144] and got["slots"][20:] == [-1, -1]
    assert got["state"] == [1, 2, 0] and got["ring"] == [9, 8, 3, 6, 5, 4]
    got = ref.plan([0, 0, 3], [17, 16, 1], [1, 0], [0, 1], [[-1, -1], [-1, -1], [2, -1]], 16, 34)
    assert got["state"] == [0, 1, 3] and got["lens"] == [0, 0, 4] and got["slots"][33] == 35


def test_reference_rotation_by_hand():
    x = np.array([[[1.0, 0.0, 0.0, 2.0]]])
    pos, axis = np.array([[1], [3]]), np.array([0, 1])
    freq = np.array([math.pi / 2, math.pi / 6])
    # halves: pairs (0, 2) by a quarter turn and (1, 3) by a quarter turn
    assert np.allclose(ref.rope(x, pos, freq, axis, False, False), [[[0, -2, 1, 0]]])
    assert np.allclose(ref.rope(x, pos, freq, axis, True, False), [[[0, 1, -2, 0]]])
    y = ref.rope(x, pos, freq, axis, True, False)
    assert np.allclose(ref.rope(y, pos, freq, axis, True, True), x)
