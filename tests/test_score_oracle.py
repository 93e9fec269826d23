"""Pins of the score-modified attention oracle and the host-side parts of the
binding, on the CPU."""

import numpy as np
import pytest
import torch

import block_sparse_attention_cross_b200 as cba
from oracle import score as osc


def _inputs(B=1, H=2, Hkv=1, Nq=7, Nk=9, d=4, seed=0):
    rng = np.random.default_rng(seed)
    return [rng.standard_normal(s) for s in ((B, H, Nq, d), (B, Hkv, Nk, d), (B, Hkv, Nk, d), (B, H, Nq, d))]


SCORES = [dict(), dict(cap=1.5), dict(slopes=np.array([0.5, 0.25])), dict(bias=True),
          dict(cap=2.0, slopes=np.array([0.1, 0.3]), bias=True)]


def _score(kw, H=2, seed=5):
    kw = dict(kw)
    if kw.pop("bias", False):
        kw["buckets"] = np.array([0, 0, 1, 2, 3, 1, 2])
        kw["table"] = np.random.default_rng(seed).standard_normal((H, 4))
    return kw


@pytest.mark.parametrize("kw", SCORES)
def test_forward_matches_torch(kw):
    q, k, v, _ = _inputs()
    kw = _score(kw)
    vis = osc.spans(1, 7, 9, causal=True, prefix=[[3]], q_start=[2])
    got = osc.score_attention(q, k, v, vis, 0.7, q_start=[2], **kw)
    tq, tk, tv = (torch.from_numpy(x) for x in (q, k, v))
    for h in range(2):
        s = 0.7 * tq[0, h] @ tk[0, 0].T
        if kw.get("cap"):
            s = kw["cap"] * torch.tanh(s / kw["cap"])
        off = torch.arange(9)[None] - (torch.arange(7)[:, None] + 2)
        if "slopes" in kw:
            s = s - float(kw["slopes"][h]) * off.abs()
        if "table" in kw:
            s = s + torch.from_numpy(kw["table"][h])[torch.from_numpy(kw["buckets"])[off.clamp(-3, 3) + 3]]
        s = s.masked_fill(~torch.from_numpy(vis[0]), float("-inf"))
        assert np.allclose(got["o"][0, h], (torch.softmax(s, 1) @ tv[0, 0]).numpy(), atol=1e-12)
        assert np.allclose(got["lse"][0, h], torch.logsumexp(s, 1).numpy(), atol=1e-12)


@pytest.mark.parametrize("kw", SCORES)
def test_gradients_match_differences(kw):
    # central differences: error h^2 (third derivatives of order 1) + 1e-16 / h
    q, k, v, do = _inputs(seed=3)
    kw = _score(kw)
    vis = osc.spans(1, 7, 9, causal=True, prefix=[[3]], q_start=[1], q_len=[6])
    g = osc.score_attention(q, k, v, vis, 0.7, q_start=[1], dout=do, **kw)

    def loss():
        return float((osc.score_attention(q, k, v, vis, 0.7, q_start=[1], **kw)["o"] * do).sum())

    rng = np.random.default_rng(1)
    pairs = [("dq", q), ("dk", k), ("dv", v)] + ([("dtable", kw["table"])] if "table" in kw else [])
    for name, x in pairs:
        for _ in range(6):
            at = tuple(int(rng.integers(n)) for n in x.shape)
            h, old = 1e-5, x[at]
            x[at] = old + h
            up = loss()
            x[at] = old - h
            down = loss()
            x[at] = old
            assert abs((up - down) / (2 * h) - g[name][at]) < 1e-7, (name, at)


def test_spans_by_hand():
    # documents [0, 2), [2, 2) (empty), [2, 5); position 5 is outside
    v = osc.spans(1, 6, 6, causal=True, docs=[[0, 2, 2, 5]], prefix=[[0, 0, 2]])[0]
    want = np.array([[1, 0, 0, 0, 0, 0], [1, 1, 0, 0, 0, 0], [0, 0, 1, 1, 0, 0], [0, 0, 1, 1, 0, 0],
                     [0, 0, 1, 1, 1, 0], [0, 0, 0, 0, 0, 0]], bool)
    assert np.array_equal(v, want)
    assert not osc.spans(1, 3, 4, kv_len=[0]).any()
    assert osc.spans(1, 3, 4, kv_len=[2], q_len=[1]).sum() == 2


@pytest.mark.parametrize("n,dist,bi", [(32, 128, True), (32, 128, False), (64, 8192, True), (4, 2, True), (2, 7, False),
                                       (256, 4096, True), (48, 1000, False)])
def test_relative_buckets_are_exact(n, dist, bi):
    got = cba.relative_buckets(n, dist, bi, device="cpu").numpy()
    want = [osc.relative_bucket(o, n, dist, bi) for o in range(-dist, dist + 1)]
    assert got.tolist() == want


def test_relative_buckets_refusals():
    for n, dist, bi in [(31, 128, True), (2, 128, True), (1, 128, False), (32, 8, True), (300, 1000, True),
                        (32, (1 << 20) + 1, True), (32, -5, True)]:
        with pytest.raises(cba.CalibattError):
            cba.relative_buckets(n, dist, bi, device="cpu")


def test_binding_refusals_without_a_gpu():
    with pytest.raises(ValueError, match="positive"):
        cba.attn_spans(0, 4, 4)
    with pytest.raises(ValueError, match="CUDA"):
        cba.attn_spans(1, 4, 4, device="cpu")
    with pytest.raises(ValueError, match="causal"):
        cba.attn_spans(1, 4, 4, prefix=[[1]], device="cuda:0")
    with pytest.raises(ValueError, match="docs"):
        cba.attn_spans(2, 4, 4, docs=[[0, 4]], device="cuda:0")
    with pytest.raises(ValueError, match="kv_len"):
        cba.attn_spans(2, 4, 4, kv_len=[4], device="cuda:0")
    with pytest.raises(ValueError, match="integers"):
        cba.attn_spans(1, 4, 4, kv_len=[4.0], device="cuda:0")
    sp = cba.AttnSpans(1, 4, 4, torch.zeros(1, 4, 2, dtype=torch.int32), torch.zeros(1, 1, 4, dtype=torch.int32),
                       torch.zeros(1, dtype=torch.int32))
    q = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="unsupported dtype"):
        cba.score_attn_fwd(q.half(), q.half(), q.half(), sp)
    with pytest.raises(TypeError, match="attn_spans"):
        cba.score_attn_fwd(q, q, q, None)
    with pytest.raises(ValueError, match="do not match"):
        cba.score_attn_fwd(q[:, :, :3], q, q, sp)
    with pytest.raises(ValueError, match="multiple of Hkv"):
        cba.score_attn_fwd(q, torch.zeros(1, 3, 4, 64, dtype=q.dtype), q, sp)
    with pytest.raises(ValueError, match="CUDA"):
        cba.score_attn_fwd(q, q, q, sp)
