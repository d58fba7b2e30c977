"""Packed attention and its gradient of batches that keep every SM busy with several units: each block takes unit
after unit from the plan, with what is left of the one before in its rings, buffers and accumulators. Against the
definition in 64 bits (packed_ref.py), and in graphs that are replayed on other documents."""
import numpy as np
import pytest
import torch

from gpu_util import fa
from test_gpu_packed import RULES, backward, batch, forward, ints, rule_of, run_both, workspace

pytestmark = pytest.mark.gpu


def units(lens, hq, hkv, rows):
    """Tiles of `rows` rows that these documents have, times the kv heads."""
    tokens = rows * hkv // hq
    return hkv * sum(-(-n // tokens) for n in lens)


def lengths(seed, docs, most):
    return [int(n) for n in np.random.default_rng(seed).integers(0, most, docs)]


def busy(lens, hq, hkv, hd):
    """Each SM has three units of the forward call and of both gradients, or more."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    fewest = min(units(lens, hq, hkv, 128 if hd == 256 else 256), units(lens, hkv, hkv, 128))
    assert fewest >= 3 * sms, (fewest, sms)


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_several_units_a_block(dtype, hd, rule):
    lens = lengths(hd, 80, 300)
    busy(lens, 6, 6, hd)
    run_both(lens, 6, 6, hd, dtype, rule_of(rule, 6, lens), gain=4.0 if "cap" in RULES[rule] else 1.0)


@pytest.mark.parametrize("rule", ["causal", "all"])
@pytest.mark.parametrize("hd", [64, 128, 256])
def test_several_units_of_shared_heads(hd, rule):
    lens = lengths(7, 75, 400)
    busy(lens, 16, 4, hd)
    run_both(lens, 16, 4, hd, "bf16", rule_of(rule, 16, lens))


@pytest.mark.parametrize("rule", ["prefix", "all", "window"])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_one_long_document_among_short_ones(dtype, hd, rule):
    """Tiles of keys that are cut into pieces beside tiles that are not."""
    lens = [*lengths(3, 40, 90), 2300, *lengths(4, 60, 90)]
    run_both(lens, 4, 2, hd, dtype, rule_of(rule, 4, lens))


def test_more_documents_than_shared_memory_holds():
    lens = lengths(9, 2100, 12)
    run_both(lens, 2, 1, 128, "f16", rule_of("all", 2, lens))


@pytest.mark.parametrize("docs", [40, 2100])
@pytest.mark.parametrize("bad", ["decreasing", "negative", "past the end"])
def test_a_planned_batch_of_bad_documents_is_flagged_and_nothing_is_written(docs, bad):
    m = fa()
    q, k, v, dout, cu = batch([3] * docs, 4, 2, 64, "bf16")
    if bad == "decreasing":
        cu[docs // 2] = cu[docs // 2 + 1] + 2
    elif bad == "negative":
        cu[0] = -1
    else:
        cu[docs] = q.shape[0] + 1
    out, lse = forward(q, k, v, cu)
    assert bool((out == -7.0).all()) and bool((lse == -7.0).all())
    assert m.get_device_error() == m.ERR_DEVICE
    made = backward(q, k, v, torch.zeros_like(out), torch.zeros_like(lse), dout, cu)
    assert all(bool((t == -7.0).all()) for t in made)
    assert m.get_device_error() == m.ERR_DEVICE
    assert m.get_device_error() == m.OK


@pytest.mark.parametrize("hd,dtype", [(64, "f16"), (128, "bf16"), (256, "f16")])
def test_planned_calls_in_a_graph_replayed_on_other_documents(hd, dtype):
    """Counters, lists and partial sums of the replay before are no part of the next one; a replay on bad documents
    writes nothing and leaves nothing behind."""
    m = fa()
    docs, T, hq, hkv = 50, 4000, 8, 4
    rule = dict(cap=20.0, win=600, sink=2)
    q, k, v, dout, _ = batch([T], hq, hkv, hd, dtype, pad=0)
    q, k, v = q.contiguous(), k.contiguous(), v.contiguous()

    def cu_of(seed, total):
        """`docs` documents, one of them with half of the tokens."""
        cuts = np.sort(np.random.default_rng(seed).integers(0, total // 2, docs - 1))
        return [0, *(int(c) for c in cuts), total]
    cu = ints(cu_of(0, T))
    out, lse = torch.empty_like(q), torch.empty(hq, T, device="cuda")
    made = [torch.empty_like(t) for t in (q, k, v)]
    ws, wsg = workspace(q, k, docs), workspace(q, k, docs, True)

    def step():
        m.packed_attn(q, k, v, out, cu, lse=lse, workspace=ws, **rule)
        m.packed_attn_grad(q, k, v, out, lse, dout, *made, cu, workspace=wsg, **rule)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed, total in ((1, T), (2, 1500), (3, T), (4, T - 1)):
        for t in (q, k, v, dout):
            t.copy_(torch.randn(t.shape, device="cuda"))
        now = cu_of(seed, total)
        want_out, want_lse = forward(q, k, v, now, **rule)
        want = backward(q, k, v, want_out, want_lse, dout, now, **rule)
        cu.copy_(ints(now))
        for t in (out, lse, *made):
            t.fill_(-7.0)
        g.replay()
        g.replay()
        assert m.get_device_error() == m.OK
        for name, a, b in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *made), (want_out, want_lse, *want)):
            assert torch.equal(a, b), (name, seed)
        cu[7] = T + 1
        for t in (out, lse, *made):
            t.fill_(-7.0)
        g.replay()
        torch.cuda.synchronize()
        assert m.get_device_error() == m.ERR_DEVICE
        assert all(bool((t == -7.0).all()) for t in (out, lse, *made))


def test_planned_calls_on_two_streams_at_once():
    m = fa()
    lens = lengths(5, 60, 300)
    q, k, v, dout, cu = batch(lens, 8, 2, 128, "bf16")
    want, wlse = forward(q, k, v, cu, cap=30.0)
    grads = backward(q, k, v, want, wlse, dout, cu, cap=30.0)
    cus = ints(cu)
    runs = [(torch.cuda.Stream(), workspace(q, k, 60), workspace(q, k, 60, True), torch.full_like(want, -7.0),
             torch.full_like(wlse, -7.0), [torch.full_like(t, -7.0) for t in grads]) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        for s, ws, wsg, out, lse, made in runs:
            m.packed_attn(q, k, v, out, cus, lse=lse, workspace=ws, cap=30.0, stream=s)
            m.packed_attn_grad(q, k, v, out, lse, dout, *made, cus, workspace=wsg, cap=30.0, stream=s)
    torch.cuda.synchronize()
    for _, _, _, out, lse, made in runs:
        assert torch.equal(out, want) and torch.equal(lse, wlse)
        assert all(torch.equal(a, b) for a, b in zip(made, grads))
    assert m.get_device_error() == m.OK
