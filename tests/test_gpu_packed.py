"""Packed attention and its gradient on the GPU against the definition in 64 bits (packed_ref.py), with
bounds from the roundings that the library makes."""
import math

import numpy as np
import pytest
import torch

import packed_ref as ref
from gpu_util import check_guards, fa, guarded

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def ints(a):
    return torch.tensor(list(a), dtype=torch.int32, device="cuda")


def batch(lens, hq, hkv, hd, dtype, seed=0, pad=3, gain=1.0, lead=0):
    """q, k, v (slices of one projection), dout and cu of documents with these lengths, padding before and behind."""
    g = torch.Generator("cuda").manual_seed(seed)
    T = lead + sum(lens) + pad
    qkv = torch.randn(T, hq + 2 * hkv, hd, device="cuda", generator=g)
    qkv[:, :hq] *= gain
    qkv = qkv.to(DT[dtype])
    dout = torch.randn(T, hq, hd, device="cuda", generator=g).to(DT[dtype])
    cu = [lead]
    for n in lens:
        cu.append(cu[-1] + n)
    return qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], dout, cu


def workspace(q, k, docs, grad=False):
    m = fa()
    size = (m.packed_attn_grad_workspace_bytes if grad else m.packed_attn_workspace_bytes)(
        docs, q.shape[0], q.shape[1], k.shape[1], q.shape[2])
    return guarded(size, torch.uint8, fill_byte=0xff)


def forward(q, k, v, cu, slopes=None, prefix=None, **rule):
    m = fa()
    out = guarded(q.shape, q.dtype, fill=-7.0)
    lse = guarded((q.shape[1], q.shape[0]), torch.float32, fill=-7.0)
    ws = workspace(q, k, len(cu) - 1)
    m.packed_attn(q, k, v, out, ints(cu), lse=lse, workspace=ws, slopes=slopes,
                  prefix=None if prefix is None else ints(prefix), **rule)
    torch.cuda.synchronize()
    check_guards(("out", out), ("lse", lse), ("workspace", ws))
    return out, lse


def backward(q, k, v, out, lse, dout, cu, slopes=None, prefix=None, **rule):
    m = fa()
    made = [guarded(t.shape, q.dtype, fill=-7.0) for t in (q, k, v)]
    ws = workspace(q, k, len(cu) - 1, True)
    m.packed_attn_grad(q, k, v, out, lse, dout, *made, ints(cu), workspace=ws, slopes=slopes,
                       prefix=None if prefix is None else ints(prefix), **rule)
    torch.cuda.synchronize()
    check_guards(("dq", made[0]), ("dk", made[1]), ("dv", made[2]), ("workspace", ws))
    return made


def close(name, got, want, err, cu):
    """Within the bound in every document, and untouched outside them."""
    live = torch.zeros(got.shape[1] if name == "lse" else got.shape[0], dtype=torch.bool, device="cuda")
    for a, b in zip(cu, cu[1:]):
        live[a:b] = True
    if name == "lse":
        got, want, err = got.T, want.T, err.T
    assert bool((got[~live] == -7.0).all()), f"{name}: padding was written"
    off = (got[live].double() - want[live]).abs()
    worst = (off / err[live].clamp(min=1e-300)).max().item() if off.numel() else 0.0
    assert bool((off <= err[live]).all()), f"{name}: {worst:.3g} of the bound"


RULES = {
    "causal": {}, "cap": dict(cap=15.0), "slopes": dict(slopes=True), "window": dict(sink=3, win=37),
    "prefix": dict(prefix=True), "all": dict(cap=8.0, slopes=True, sink=1, win=50, prefix=True), "narrow": dict(win=1),
}


def rule_of(name, hq, lens):
    rule = dict(RULES[name])
    if rule.get("slopes"):
        rule["slopes"] = torch.exp2(-torch.arange(1, hq + 1, device="cuda") * 0.7).float()
    if rule.get("prefix"):
        rule["prefix"] = [(7 * i * i + 2) % (n + 9) if n else 3 for i, n in enumerate(lens)]
    return rule


LENS = [[1], [5], [128], [129, 0, 1, 127], [300, 64, 0, 33, 257]]


def run_both(lens, hq, hkv, hd, dtype, rule, seed=1, **kw):
    q, k, v, dout, cu = batch(lens, hq, hkv, hd, dtype, seed, **kw)
    want = ref.packed(q, k, v, cu, dout=dout, **rule)
    out, lse = forward(q, k, v, cu, **rule)
    close("out", out, want["out"], want["out_err"], cu)
    close("lse", lse, want["lse"], want["lse_err"], cu)
    made = backward(q, k, v, out, lse, dout, cu, **rule)
    for name, t in zip(("dq", "dk", "dv"), made):
        close(name, t, want[name], want[name + "_err"], cu)
    assert fa().get_device_error() == fa().OK


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_lengths(dtype, hd, lens):
    run_both(lens, 4, 2, hd, dtype, {})


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_rules(dtype, hd, rule):
    lens = [150, 1, 0, 283, 40]
    run_both(lens, 8, 2, hd, dtype, rule_of(rule, 8, lens), gain=4.0 if "cap" in RULES[rule] else 1.0)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 3), (2, 1), (8, 1), (16, 1), (32, 2)])
@pytest.mark.parametrize("hd", [64, 128, 256])
def test_groups(hd, hq, hkv):
    lens = [77, 5, 0, 140]
    run_both(lens, hq, hkv, hd, "bf16", rule_of("all", hq, lens))


def test_many_documents():
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(0, 9, 2500)]  # more documents than shared memory holds
    run_both(lens, 2, 1, 64, "bf16", {}, lead=2)


def test_long_document():
    run_both([4100], 2, 1, 128, "f16", rule_of("slopes", 2, [4100]))
    run_both([2500], 1, 1, 256, "bf16", dict(sink=130, win=700))


def test_scale():
    run_both([90, 33], 4, 4, 64, "bf16", dict(scale=0.31))
    run_both([90, 33], 4, 4, 64, "f16", dict(scale=0.31, cap=3.0))


def test_large_scores():
    """Scores of hundreds: the reference moves, and the first weights vanish beside later ones."""
    run_both([260], 2, 1, 64, "bf16", {}, gain=30.0)
    run_both([260], 2, 1, 64, "f16", dict(cap=300.0), gain=30.0)


@pytest.mark.parametrize("size", [2.0 ** -14, 2.0 ** -6, 2.0 ** 9])
def test_binary16_gradients_of_any_size(size):
    """A dout of any magnitude keeps its precision; of another power of two it gives the same bits."""
    q, k, v, dout, cu = batch([150, 70], 4, 2, 64, "f16")
    out, lse = forward(q, k, v, cu)
    # (a product below 2^-14 is rounded, and what comes of it may round every t and every weight's product
    # the other way: not the scaled gradient itself but the definition's, for this dout, has to be met)
    want = ref.packed(q, k, v, cu, dout=dout * size)
    made = backward(q, k, v, out, lse, dout * size, cu)
    for name, t in zip(("dq", "dk", "dv"), made):
        close(name, t, want[name], want[name + "_err"], cu)
    if size > 1:  # a power of two, exact everywhere
        base = backward(q, k, v, out, lse, dout, cu)
        for name, a, b in zip(("dq", "dk", "dv"), made, base):
            normal = b.abs() >= 2.0 ** -14
            normal[:cu[0]] = normal[cu[-1]:] = False
            assert torch.equal(a[normal], (b * size)[normal]), name


@pytest.mark.parametrize("dtype,hd", [("bf16", 64), ("f16", 128), ("bf16", 256)])
def test_other_documents_and_padding_may_hold_anything(dtype, hd):
    lens = [70, 130, 45]
    q, k, v, dout, cu = batch(lens, 4, 2, hd, dtype, pad=9, lead=5)
    out, lse = forward(q, k, v, cu)
    made = backward(q, k, v, out, lse, dout, cu)
    bad = torch.tensor([float("nan"), float("inf"), -float("inf")], device="cuda", dtype=DT[dtype])
    keep = torch.zeros(q.shape[0], dtype=torch.bool, device="cuda")
    keep[cu[1]:cu[2]] = True
    for t in (q, k, v, dout, out):
        junk = bad[torch.arange(t.numel(), device="cuda") % 3].view(t.shape)
        t.copy_(torch.where(keep[:, None, None], t, junk))
    lse.copy_(torch.where(keep, lse, torch.nan))
    out2, lse2 = forward(q, k, v, cu)
    assert torch.equal(out2[keep], out[keep]) and torch.equal(lse2[:, keep], lse[:, keep])
    for name, a, b in zip(("dq", "dk", "dv"), backward(q, k, v, out, lse, dout, cu), made):
        assert torch.equal(a[keep], b[keep]), name


@pytest.mark.parametrize("rule", [*RULES, "capped prefix"])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_neighbours_of_a_document_change_no_bit(dtype, hd, rule):
    """Documents of odd and even lengths between others that hold NaN, infinities or the largest values, under every
    rule (the last one: capped scores, and a prefix of the whole document)."""
    largest = torch.finfo(DT[dtype]).max
    for n, hq, hkv in ((1, 2, 2), (37, 4, 1), (127, 2, 2), (129, 4, 1), (130, 2, 2), (131, 8, 2)):
        lens = [70, n, 45]
        given = dict(cap=20.0, prefix=lens) if rule == "capped prefix" else rule_of(rule, hq, lens)
        q, k, v, dout, cu = batch(lens, hq, hkv, hd, dtype, pad=9, lead=5)
        out, lse = forward(q, k, v, cu, **given)
        made = backward(q, k, v, out, lse, dout, cu, **given)
        keep = torch.zeros(q.shape[0], dtype=torch.bool, device="cuda")
        keep[cu[1]:cu[2]] = True
        for junk in ((math.nan, math.inf, -math.inf), (largest, -largest, 0.0)):
            bad = torch.tensor(junk, device="cuda", dtype=DT[dtype])
            q2, k2, v2, dout2, out2 = (
                torch.where(keep[:, None, None], t, bad[torch.arange(t.numel(), device="cuda") % 3].view(t.shape))
                for t in (q, k, v, dout, out))
            lse2 = torch.where(keep, lse, torch.nan)
            again = forward(q2, k2, v2, cu, **given)
            assert torch.equal(again[0][keep], out[keep]) and torch.equal(again[1][:, keep], lse[:, keep]), (n, junk)
            for name, a, b in zip(("dq", "dk", "dv"), backward(q2, k2, v2, out2, lse2, dout2, cu, **given), made):
                assert torch.equal(a[keep], b[keep]), (name, n, junk)
    assert fa().get_device_error() == fa().OK


def test_gradient_against_differences():
    """The gradient along a direction against central differences of the definition in 64 bits."""
    lens, rule = [60, 33], dict(cap=4.0, sink=2, win=20, prefix=[9, 0])
    slopes = torch.tensor([0.3, 0.05], device="cuda")
    q, k, v, dout, cu = batch(lens, 2, 1, 64, "f16", pad=0)
    out, lse = forward(q, k, v, cu, slopes=slopes, **rule)
    made = backward(q, k, v, out, lse, dout, cu, slopes=slopes, **rule)

    def loss(q, k, v):
        total = 0.0
        for d in range(2):
            at = slice(cu[d], cu[d + 1])
            for h in range(2):
                r = ref.document(q[at, h], k[at, 0], v[at, 0], float(slopes[h]), prefix=rule["prefix"][d],
                                 sink=2, win=20, cap=4.0)
                total += (r["out"] * dout[at, h].double()).sum().item()
        return total
    g = torch.Generator("cuda").manual_seed(9)
    wide = [t.double() for t in (q, k, v)]
    want = ref.packed(q, k, v, cu, slopes=slopes, dout=dout, **rule)
    for i, name in enumerate(("dq", "dk", "dv")):
        step = torch.randn(wide[i].shape, device="cuda", generator=g, dtype=torch.float64)
        h = 1e-4
        ends = [loss(*[t + (s * h * step if n == i else 0) for n, t in enumerate(wide)]) for s in (1, -1)]
        slope = (ends[0] - ends[1]) / (2 * h)
        along = (made[i].double() * step).sum().item()
        # the bound of every value along the step; central differences are off by h^2 of the third derivative
        tol = (want[name + "_err"] * step.abs()).sum().item() + 1e-5 * (1 + abs(slope))
        assert abs(along - slope) <= tol, (name, along, slope)


def test_equal_calls_give_equal_bits():
    q, k, v, dout, cu = batch([500, 1, 700, 90], 8, 2, 128, "bf16")
    first = None
    for _ in range(4):
        out, lse = forward(q, k, v, cu)
        made = [t.clone() for t in (out, lse, *backward(q, k, v, out, lse, dout, cu))]
        first = first or made
        assert all(torch.equal(a, b) for a, b in zip(made, first))


def test_strides_of_outputs():
    """Results into slices of wider tensors, whose other columns stay as they are."""
    m = fa()
    q, k, v, dout, cu = batch([90, 41], 4, 2, 64, "bf16")
    out, lse = forward(q, k, v, cu)
    want = backward(q, k, v, out, lse, dout, cu)
    T = q.shape[0]
    wide = torch.full((T, 4 + 2 + 2 + 1 + 4, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    dq, dk, dv, o = wide[:, :4], wide[:, 4:6], wide[:, 6:8], wide[:, 9:]
    m.packed_attn(q, k, v, o, ints(cu), workspace=workspace(q, k, 2))
    m.packed_attn_grad(q, k, v, o, lse, dout, dq, dk, dv, ints(cu), workspace=workspace(q, k, 2, True))
    n = cu[-1]
    for a, b in zip((o, dq, dk, dv), (out, *want)):
        assert torch.equal(a[:n], b[:n])
    assert bool((wide[:, 8] == 5.0).all()) and bool((wide[n:] == 5.0).all())


@pytest.mark.parametrize("cu", [[0, 50, 40, 90], [-1, 50, 60, 90], [0, 50, 60, 94], [3, 1, 2, 0]], ids=str)
def test_bad_documents_are_flagged_and_nothing_is_written(cu):
    m = fa()
    q, k, v, dout, _ = batch([90], 4, 2, 64, "bf16", pad=3)
    out, lse = forward(q, k, v, cu)
    assert bool((out == -7.0).all()) and bool((lse == -7.0).all())
    assert m.get_device_error() == m.ERR_DEVICE
    made = backward(q, k, v, torch.zeros_like(out), torch.zeros_like(lse), dout, cu)
    assert all(bool((t == -7.0).all()) for t in made)
    assert m.get_device_error() == m.ERR_DEVICE
    assert m.get_device_error() == m.OK


def test_prefix_out_of_range_is_cut():
    q, k, v, dout, cu = batch([40, 25], 4, 2, 64, "bf16")
    a, _ = forward(q, k, v, cu, prefix=[-5, 1 << 30])
    b, _ = forward(q, k, v, cu, prefix=[0, 25])
    assert torch.equal(a, b)


def test_graphs_and_streams():
    """Two captured training steps with workspaces of their own, replayed on new inputs and documents, beside
    calls on another stream."""
    m = fa()
    q, k, v, dout, cu = batch([200, 100], 4, 2, 128, "bf16")
    q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    docs = ints(cu)
    lse = torch.empty(4, q.shape[0], device="cuda")

    def step(ws, wsg, out, grads):
        m.packed_attn(q, k, v, out, docs, lse=lse, workspace=ws, cap=20.0)
        m.packed_attn_grad(q, k, v, out, lse, dout, *grads, docs, workspace=wsg, cap=20.0)
    graphs, results = [], []
    for _ in range(2):
        ws, wsg = workspace(q, k, 2), workspace(q, k, 2, True)
        out = torch.full_like(q, -7.0)
        grads = [torch.full_like(t, -7.0) for t in (q, k, v)]
        step(ws, wsg, out, grads)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(ws, wsg, out, grads)
        graphs.append(g)
        results.append((ws, wsg, out, grads))
    for seed, lens in ((5, [200, 100]), (6, [7, 250])):
        q2, k2, v2, d2, cu2 = batch(lens, 4, 2, 128, "bf16", seed=seed, pad=303 - sum(lens))
        for a, b in ((q, q2), (k, k2), (v, v2), (dout, d2)):
            a.copy_(b)
        docs.copy_(ints(cu2))
        want = ref.packed(q, k, v, cu2, dout=dout, cap=20.0)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            graphs[0].replay()
        torch.cuda.current_stream().wait_stream(side)
        graphs[1].replay()
        torch.cuda.synchronize()
        for _, _, out, grads in results:
            n = cu2[-1]
            for name, t in zip(("out", "dq", "dk", "dv"), (out, *grads)):
                off = (t[:n].double() - want[name][:n]).abs()
                assert bool((off <= want[name + "_err"][:n]).all()), name
    assert m.get_device_error() == m.OK


def test_two_streams_at_once():
    m = fa()
    q, k, v, dout, cu = batch([900, 300], 8, 2, 128, "bf16")
    want, wlse = forward(q, k, v, cu)
    grads = backward(q, k, v, want, wlse, dout, cu)
    docs = ints(cu)
    runs = []
    for _ in range(2):
        runs.append((torch.cuda.Stream(), workspace(q, k, 2), workspace(q, k, 2, True), torch.full_like(want, -7.0),
                     torch.full_like(wlse, -7.0), [torch.full_like(t, -7.0) for t in grads]))
    torch.cuda.synchronize()
    for _ in range(3):
        for s, ws, wsg, out, lse, made in runs:
            m.packed_attn(q, k, v, out, docs, lse=lse, workspace=ws, stream=s)
            m.packed_attn_grad(q, k, v, out, lse, dout, *made, docs, workspace=wsg, stream=s)
    torch.cuda.synchronize()
    for _, _, _, out, lse, made in runs:
        assert torch.equal(out, want) and torch.equal(lse, wlse)
        assert all(torch.equal(a, b) for a, b in zip(made, grads))


def test_refusals_of_the_binding():
    m = fa()
    q, k, v, dout, cu = batch([40], 4, 2, 64, "bf16")
    out, lse, docs = torch.empty_like(q), torch.empty(4, q.shape[0], device="cuda"), ints(cu)
    ws = workspace(q, k, 1)
    call = lambda **kw: m.packed_attn(**{**dict(q=q, k=k, v=v, out=out, cu_docs=docs, workspace=ws), **kw})  # noqa: E731
    for bad in (dict(q=q.cpu()), dict(k=k.half()), dict(v=v[:-1]), dict(out=out[:, :2]), dict(cu_docs=docs.long()),
                dict(cu_docs=docs.cpu()), dict(cu_docs=docs[:0]), dict(prefix=ints([1, 2])), dict(slopes=torch.ones(3, device="cuda")),
                dict(lse=lse[:2]), dict(q=q.transpose(1, 2)), dict(workspace=ws.float())):
        with pytest.raises(ValueError):
            call(**bad)
    for bad, status in ((dict(cap=-1.0), m.ERR_INVALID), (dict(cap=math.nan), m.ERR_INVALID), (dict(sink=-1), m.ERR_INVALID),
                        (dict(workspace=ws[:256]), m.ERR_WORKSPACE), (dict(out=q), m.ERR_INVALID),
                        (dict(q=q.float(), k=k.float(), v=v.float(), out=out.float()), m.ERR_UNSUPPORTED)):
        with pytest.raises(m.FAError) as e:
            call(**bad)
        assert e.value.status == status, bad
    with pytest.raises(m.FAError):
        m.packed_attn_grad(q, k, v, out, lse, dout, dout, torch.empty_like(k), torch.empty_like(v), docs,
                           workspace=workspace(q, k, 1, True))
    assert m.get_device_error() == m.OK


def test_no_tokens_and_no_documents():
    m = fa()
    q, k, v, dout, cu = batch([40], 4, 2, 64, "bf16")
    out = torch.full_like(q, -7.0)
    m.packed_attn(q, k, v, out, ints([0]), workspace=workspace(q, k, 0))
    m.packed_attn(q[:0], k[:0], v[:0], out[:0], ints([0, 0]), workspace=workspace(q[:0], k, 1))
    m.packed_attn(q, k, v, out, ints([5, 5, 5]), workspace=workspace(q, k, 2))
    torch.cuda.synchronize()
    assert bool((out == -7.0).all()) and m.get_device_error() == m.OK
