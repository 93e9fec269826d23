"""Score-modified attention as part of the autograd graph: the gradients are
score_attn_bwd's, bit for bit, and what has none raises instead of losing it."""

import pytest
import torch

import block_sparse_attention_cross_b200 as cba
from tests._score_util import Case

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _leaves(c, names=("q", "k", "v", "table")):
    t = {n: c.gpu(getattr(c, n)) for n in ("q", "k", "v", "table")}
    for n in names:
        if t[n] is not None:
            t[n].requires_grad_()
    kw = c.score_kw()
    kw["table"] = t["table"]
    return t, kw


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kw", [dict(), dict(cap=4.0, slopes=True, buckets=8, distance=30, causal=True, layout="bnhd", Hkv=2)])
def test_gradients_are_the_backwards(dtype, kw):
    c = Case(B=2, H=4, Nq=150, d=64, dtype=dtype, **kw)
    want = c.run(True)
    t, skw = _leaves(c)
    o, lse = cba.score_attn_fwd(t["q"], t["k"], t["v"], c.spans(), return_lse=True, **skw)
    assert o.requires_grad and torch.equal(o, want["o"]) and torch.equal(lse, want["lse"])
    o.backward(c.gpu(c.do))
    for n in ("q", "k", "v", "table"):
        if t[n] is not None:
            assert torch.equal(t[n].grad, want["d" + n]), n


@pytest.mark.parametrize("dtype", [BF, F32])
def test_expanded_gradient_and_single_leaves(dtype):
    c = Case(B=1, H=2, Nq=70, d=64, dtype=dtype, cap=3.0, buckets=6, distance=20)
    c.do = torch.ones_like(c.do)
    want = c.run(True)
    for n in ("q", "k", "v", "table"):
        t, skw = _leaves(c, (n,))
        cba.score_attn_fwd(t["q"], t["k"], t["v"], c.spans(), **skw).sum().backward()
        assert torch.equal(t[n].grad, want["d" + n]), n
        assert all(t[m].grad is None for m in t if m != n)


def test_no_graph_without_need():
    c = Case(H=2, Nq=40, d=64, buckets=4, distance=9)
    t, skw = _leaves(c)
    with torch.no_grad():
        assert not cba.score_attn_fwd(t["q"], t["k"], t["v"], c.spans(), **skw).requires_grad
    t, skw = _leaves(c, ())
    assert not cba.score_attn_fwd(t["q"], t["k"], t["v"], c.spans(), **skw).requires_grad


def test_callers_buffers_join_the_graph():
    c = Case(H=2, Nq=40, d=64)
    want = c.run(True)
    t, skw = _leaves(c)
    out, lse = torch.empty_like(want["o"]), torch.empty_like(want["lse"])
    r = cba.score_attn_fwd(t["q"], t["k"], t["v"], c.spans(), out=out, lse=lse, **skw)
    assert r.data_ptr() == out.data_ptr() and torch.equal(lse, want["lse"])
    r.backward(c.gpu(c.do))
    assert torch.equal(t["k"].grad, want["dk"])
    assert not out.requires_grad and not lse.requires_grad
    # the buffers serve the next step; a graph that saved what they held says so
    r = cba.score_attn_fwd(t["q"], t["k"], t["v"], c.spans(), out=out, lse=lse, **skw)
    cba.score_attn_fwd(t["q"], t["k"], t["v"], c.spans(), out=out, lse=lse, **skw).backward(c.gpu(c.do))
    assert torch.equal(t["k"].grad, 2 * want["dk"])
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        r.backward(c.gpu(c.do))


def test_what_has_no_gradient_raises():
    c = Case(H=2, Nq=40, d=64, slopes=True)
    t, skw = _leaves(c)
    o, lse = cba.score_attn_fwd(t["q"], t["k"], t["v"], c.spans(), return_lse=True, **skw)
    with pytest.raises(RuntimeError, match="LSE"):
        (o.float().sum() + lse.sum()).backward()
    skw["slopes"] = skw["slopes"].clone().requires_grad_()
    o = cba.score_attn_fwd(c.gpu(c.q), c.gpu(c.k), c.gpu(c.v), c.spans(), **skw)
    with pytest.raises(RuntimeError, match="slopes"):
        o.sum().backward()
    t, skw = _leaves(c)
    o = cba.score_attn_fwd(t["q"], t["k"], t["v"], c.spans(), **skw)
    g, = torch.autograd.grad(o.float().sum(), t["q"], create_graph=True)
    with pytest.raises(RuntimeError):
        g.float().sum().backward()


def test_training_step_captured():
    # a projection before the attention, forward and backward in one graph, replayed on other inputs
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(1, 130, 128, device="cuda", generator=g).to(BF)
    w = (torch.randn(128, 3 * 128, device="cuda", generator=g) * 0.1).to(BF).requires_grad_()
    sp = cba.attn_spans(1, 130, 130, causal=True)

    def step():
        q, k, v = ((x @ w).view(1, 130, 3, 2, 64)[:, :, i].transpose(1, 2) for i in range(3))
        o = cba.score_attn_fwd(q, k, v, sp, cap=20.0)
        dw, = torch.autograd.grad(o.float().pow(2).sum(), w)
        return o.detach(), dw

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (2, 3):
        x.copy_(torch.randn(1, 130, 128, device="cuda", generator=g.manual_seed(seed)).to(BF))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
