"""Packed attention, scored paged attention and the append that rotates, without a GPU: what they refuse before any
launch, workspace sizes, and pins of the reference that the GPU tests compare with."""
import math

import numpy as np
import pytest
import torch

import packed_ref as ref


@pytest.fixture(scope="module")
def fa():
    from causal_gqa_flash_attn_gb300 import build
    build.build()
    import causal_gqa_flash_attn_gb300 as fa
    fa.lib()
    return fa


def caller(fn, names, **base):
    """A call by keyword whose other arguments are valid (pointers are multiples of 16, never read)."""
    def call(**kw):
        a = {**base, **kw}
        assert set(a) == set(names), set(a) ^ set(names)
        return fn(*[a[n] for n in names])
    return call


SHARED = dict(type=2, cu=16, prefix=None, docs=3, T=40, hq=8, hkv=2, hd=64, sink=0, win=0, scale=0.0, cap=0.0, slopes=None,
              ws=16, wsb=1 << 40, stream=None)
RULES = (dict(type=3), dict(type=-1), dict(docs=-1), dict(T=-1), dict(hq=0), dict(hkv=0), dict(hq=9), dict(hd=16),
         dict(hd=100), dict(sink=-1), dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf), dict(cap=-1.0),
         dict(cap=math.nan), dict(cap=math.inf), dict(cap=1e-39), dict(cu=None), dict(cu=18), dict(prefix=18), dict(slopes=18),
         dict(ws=None), dict(ws=24))
UNSUPPORTED = (dict(type=0), dict(cap=4097.0), dict(hd=96), dict(hd=32), dict(hq=24), dict(hq=64, hkv=2), dict(docs=65537),
               dict(T=(1 << 26) + 1), dict(T=1 << 26, hq=32, hkv=2))


def test_packed_refusals(fa):
    names = ("q k v out lse type qs ks vs os cu prefix docs T hq hkv hd sink win scale cap slopes ws wsb stream").split()
    call = caller(fa.lib().fa_packed_attn, names, q=16, k=32, v=48, out=64, lse=16, qs=512, ks=128, vs=128, os=512,
                  **SHARED)
    for bad in RULES + (dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(q=24), dict(out=72), dict(lse=18),
                        dict(qs=504), dict(ks=120), dict(vs=132), dict(os=0), dict(qs=516), dict(ks=1 << 36), dict(out=16),
                        dict(out=32), dict(out=48)):
        assert call(**bad) == fa.ERR_INVALID, bad
    for bad in UNSUPPORTED:
        assert call(**bad) == fa.ERR_UNSUPPORTED, bad
    need = fa.packed_attn_workspace_bytes(3, 40, 8, 2, 64)
    assert call(wsb=need - 1) == fa.ERR_WORKSPACE
    assert call(T=0) == fa.OK and call(docs=0) == fa.OK


def test_packed_grad_refusals(fa):
    names = ("q k v out lse dout dq dk dv type qs ks vs os dos dqs dks dvs cu prefix docs T hq hkv hd sink win scale cap "
             "slopes ws wsb stream").split()
    call = caller(fa.lib().fa_packed_attn_grad, names, q=16, k=32, v=48, out=64, lse=16, dout=80, dq=96, dk=112, dv=128,
                  qs=512, ks=128, vs=128, os=512, dos=512, dqs=512, dks=128, dvs=128, **SHARED)
    for bad in RULES + tuple({n: None} for n in "q k v out lse dout dq dk dv".split()) + (
            dict(lse=18), dict(dq=104), dict(dos=504), dict(dks=64), dict(dvs=129), dict(dq=16), dict(dk=32), dict(dv=80),
            dict(dq=112), dict(dk=128), dict(dv=96)):
        assert call(**bad) == fa.ERR_INVALID, bad
    for bad in UNSUPPORTED:
        assert call(**bad) == fa.ERR_UNSUPPORTED, bad
    need = fa.packed_attn_grad_workspace_bytes(3, 40, 8, 2, 64)
    assert call(wsb=need - 1) == fa.ERR_WORKSPACE
    assert call(T=0) == fa.OK and call(docs=0) == fa.OK


def test_packed_workspaces(fa):
    for size in (fa.packed_attn_workspace_bytes, fa.packed_attn_grad_workspace_bytes):
        assert size(3, 40, 8, 2, 96) == 0 and size(-1, 40, 8, 2, 64) == 0 and size(1, 40, 9, 2, 64) == 0
        assert 0 < size(0, 0, 8, 2, 64) < size(1, 1, 8, 2, 64) <= size(1, 5000, 8, 2, 64)
    # the gradient keeps two numbers for each row, and partial sums, 48 MiB at most
    rows = 8192 * 16
    assert 8 * rows <= fa.packed_attn_grad_workspace_bytes(1, 8192, 16, 2, 256) < 16 * rows + (48 << 20)
    assert fa.packed_attn_grad_workspace_bytes(1, 300, 4, 4, 64) < 1 << 18
    for n in (1, 200, 5000, 1 << 20):
        for docs in (1, 7, 5000):
            for hq, hkv, hd in ((1, 1, 64), (16, 1, 128), (32, 8, 256)):
                assert fa.packed_attn_workspace_bytes(docs, n, hq, hkv, hd) < (1 << 20) + 8 * n * hq + 512 * docs
                assert (fa.packed_attn_grad_workspace_bytes(docs, n, hq, hkv, hd)
                        < (50 << 20) + 16 * n * hq + 2048 * hkv * docs)


def test_packed_factors_of_scores_are_finite(fa):
    """scale * log2 e, and 2 * scale * log2 e / cap where scores are capped: an infinite one times a score of 0 is a
    NaN, and so is 0 times the -inf of a masked score, where a factor below the normal range is flushed; such calls
    are refused. Without a workspace, what is taken goes no further than its absence."""
    names = ("q k v out lse type qs ks vs os cu prefix docs T hq hkv hd sink win scale cap slopes ws wsb stream").split()
    call = caller(fa.lib().fa_packed_attn, names, q=16, k=32, v=48, out=64, lse=16, qs=512, ks=128, vs=128, os=512,
                  **SHARED)
    names = ("q k v out lse dout dq dk dv type qs ks vs os dos dqs dks dvs cu prefix docs T hq hkv hd sink win scale cap "
             "slopes ws wsb stream").split()
    grad = caller(fa.lib().fa_packed_attn_grad, names, q=16, k=32, v=48, out=64, lse=16, dout=80, dq=96, dk=112, dv=128,
                  qs=512, ks=128, vs=128, os=512, dos=512, dqs=512, dks=128, dvs=128, **SHARED)
    for f in (call, grad):
        for bad in (dict(scale=9e37), dict(scale=1e3, cap=1e-36), dict(scale=8.0, cap=9e-38), dict(scale=9e37, cap=1.0),
                    dict(scale=1.1e-38), dict(scale=1e-45), dict(scale=1.1e-38, cap=3.0)):
            assert f(wsb=0, **bad) == fa.ERR_INVALID, bad
        for good in (dict(scale=8e37), dict(scale=1.2e-38), dict(scale=1e3, cap=2e-35), dict(cap=2e-38), dict(scale=8.0, cap=1e-37),
                     dict(scale=8e37, cap=4096.0)):
            assert f(wsb=0, **good) == fa.ERR_WORKSPACE, good


def test_scored_refusals(fa):
    names = ("q out lse type qs os cu lens table max_pages pages n_pages rows reqs T hq hkv hd sink win scale cap slopes "
             "ws wsb stream").split()
    call = caller(fa.lib().fa_paged_attn_scored, names, q=16, out=32, lse=16, type=2, qs=512, os=512, cu=16, lens=16,
                  table=16, max_pages=4, pages=16, n_pages=9, rows=16, reqs=3, T=4, hq=8, hkv=2, hd=64, sink=0, win=0,
                  scale=0.0, cap=5.0, slopes=16, ws=16, wsb=1 << 40, stream=None)
    for bad in (dict(cap=-1.0), dict(cap=math.nan), dict(cap=math.inf), dict(slopes=18), dict(q=None), dict(rows=24),
                dict(out=16), dict(scale=-1.0), dict(type=3), dict(sink=-1)):
        assert call(**bad) == fa.ERR_INVALID, bad
    assert call(cap=1e-39) == fa.ERR_INVALID
    assert call(hd=96) == fa.ERR_UNSUPPORTED and call(cap=5000.0) == fa.ERR_UNSUPPORTED
    assert call(T=0) == fa.OK


def test_rope_append_refusals(fa):
    names = ("q q_out k v type T hq hkv hd rd qs qos ks vs pos pos_stride axes table adjacent slots pages n_pages rows "
             "stream").split()
    call = caller(fa.lib().fa_rope_append, names, q=16, q_out=32, k=48, v=64, type=2, T=4, hq=8, hkv=2, hd=64, rd=64, qs=512,
                  qos=512, ks=128, vs=128, pos=16, pos_stride=4, axes=1, table=16, adjacent=0, slots=16, pages=16, n_pages=9,
                  rows=16, stream=None)
    for bad in (dict(type=3), dict(T=-1), dict(hq=-1), dict(hq=65537), dict(hkv=0), dict(hd=40), dict(rd=0), dict(rd=7),
                dict(rd=66), dict(axes=0), dict(axes=9), dict(rows=24), dict(n_pages=0), dict(q=None), dict(q_out=None),
                dict(q=24), dict(q_out=40), dict(qs=504), dict(qos=516), dict(q=32, qs=520), dict(k=None), dict(v=None),
                dict(k=56), dict(ks=120), dict(vs=132), dict(pos=None), dict(pos=18), dict(pos_stride=3), dict(table=None),
                dict(table=24), dict(slots=None), dict(slots=18), dict(pages=None), dict(pages=24)):
        assert call(**bad) == fa.ERR_INVALID, bad
    for bad in (dict(hd=96), dict(hkv=65536), dict(T=(1 << 30) + 1)):
        assert call(**{"pos_stride": 1 << 31, **bad}) == fa.ERR_UNSUPPORTED, bad
    assert call(T=0) == fa.OK


def test_binding_refuses_tensors_of_the_host(fa):
    q, k = torch.zeros(4, 8, 64).bfloat16(), torch.zeros(4, 2, 64).bfloat16()
    i, ws = torch.zeros(2, dtype=torch.int32), torch.zeros(1 << 16, dtype=torch.uint8)
    with pytest.raises(ValueError):
        fa.packed_attn(q, k, k, q, i, workspace=ws)
    with pytest.raises(ValueError):
        fa.packed_attn_grad(q, k, k, q, torch.zeros(8, 4), q, q, k, k, i, workspace=ws)
    with pytest.raises(ValueError):
        fa.rope_append(q, k, k, q, i, torch.zeros(32, 4, dtype=torch.int32), i, ws, page_rows=16)


# ------------------------------------------------------- pins of the reference

def test_reference_sees():
    assert ref.seen(4).tolist() == [[j <= i for j in range(4)] for i in range(4)]
    assert ref.seen(4, prefix=2, sink=0, win=1).int().tolist() == [[1, 1, 0, 0], [1, 1, 0, 0], [1, 1, 1, 0], [1, 1, 0, 1]]
    assert ref.seen(5, sink=1, win=2).int().tolist() == [[1, 0, 0, 0, 0], [1, 1, 0, 0, 0], [1, 1, 1, 0, 0], [1, 0, 1, 1, 0],
                                                         [1, 0, 0, 1, 1]]


def test_reference_by_hand():
    """Two keys, scores a and b: weights 1 / (1 + e^(b - a)) and the rest."""
    q = torch.tensor([[1.0], [2.0]], dtype=torch.float64)
    k = torch.tensor([[0.5], [-1.0]], dtype=torch.float64)
    v = torch.tensor([[3.0], [7.0]], dtype=torch.float64)
    r = ref.document(q, k, v, 0.25, scale=1.0)
    assert r["out"][0, 0] == 3.0 and r["lse"][0] == 0.5
    a, b = 1.0 - 0.25, -2.0
    w = math.exp(a) / (math.exp(a) + math.exp(b))
    assert abs(r["out"][1, 0] - (3 * w + 7 * (1 - w))) < 1e-12
    r = ref.document(q, k, v, 0.0, scale=1.0, cap=1.5)
    a, b = 1.5 * math.tanh(1 / 1.5), 1.5 * math.tanh(-2 / 1.5)
    assert abs(r["lse"][1] - math.log(math.exp(a) + math.exp(b))) < 1e-12


def test_reference_gradient_against_differences():
    g = torch.Generator().manual_seed(0)
    q, k, v, do = (torch.randn(9, 8, generator=g, dtype=torch.float64) for _ in range(4))
    rule = dict(prefix=3, sink=1, win=4, cap=1.3)
    r = ref.document(q, k, v, 0.2, dout=do, **rule)
    for name, x in (("dq", q), ("dk", k), ("dv", v)):
        for at in ((0, 0), (4, 3), (8, 7)):
            ends = []
            for s in (1e-6, -1e-6):
                y = x.clone()
                y[at] += s
                t = [y if z is x else z for z in (q, k, v)]
                ends.append((ref.document(*t, 0.2, **rule)["out"] * do).sum())
            assert abs((ends[0] - ends[1]) / 2e-6 - r[name][at]) < 1e-7, (name, at)
    assert np.isfinite(r["t_err"].numpy()).all()
