"""Score-modified attention on the GPU against the float64 oracle, within the
narrow limits of tests/_score_check.py (which refuse a missing term, tile or
group of rows)."""

import numpy as np
import pytest
import torch

import block_sparse_attention_cross_b200 as cba
from tests._score_check import Narrow

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kw", [
    dict(Nq=1, d=64), dict(Nq=129, d=128), dict(Nq=300, d=64), dict(Nq=300, d=128, cap=5.0),
    dict(Nq=333, H=3, cap=50.0, gain=8.0), dict(Nq=333, H=3, slopes=True), dict(Nq=333, H=3, buckets=32, distance=200),
    dict(Nq=333, H=3, buckets=8, distance=1000, bidirectional=False, causal=True),
    dict(Nq=333, H=3, cap=2.0, slopes=True, buckets=6, distance=40, causal=True),
    dict(Nq=333, H=3, buckets=256, distance=300, cap=4.0),
    dict(Nq=260, d=64, scale=4.0, gain=6.0), dict(Nq=260, d=64, scale=4.0, gain=6.0, cap=100.0),
])
def test_scores(dtype, kw):
    Narrow(dtype=dtype, **kw).verify()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kw", [
    dict(causal=True, prefix=[[40], [300]]),
    dict(docs=[[0, 100, 101, 270], [3, 3, 130, 260]], causal=True, prefix=[[1, 1, 64], [5, 100, 2]]),
    dict(kv_len=[0, 129], q_len=[0, 200]),
])
def test_masks_and_shared_heads(dtype, kw):
    Narrow(B=2, H=4, Hkv=2, Nq=270, d=64, dtype=dtype, cap=3.0, slopes=True, buckets=12, distance=50, **kw).verify()
    Narrow(B=2, H=10, Hkv=2, Nq=270, d=128, dtype=dtype, layout="bnhd", **kw).verify()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_few_queries(dtype):
    lens = [1111, 400, 1]
    for kw in (dict(), dict(cap=5.0, slopes=True, buckets=16, distance=600)):
        Narrow(B=3, H=16, Hkv=4, Nq=5, Nk=1111, d=128, dtype=dtype, causal=True, kv_len=lens, q_start=[max(0, n - 5) for n in lens],
               q_len=[min(n, 5) for n in lens], **kw).verify()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kw", [dict(), dict(cap=4.0, slopes=True, buckets=16, distance=70)])
def test_calibrated_mask(dtype, kw):
    m = (np.random.default_rng(7).random((2, 4, 4)) < 0.5).astype(np.uint8)
    m[1, 2] = 0
    Narrow(H=2, Nq=450, d=128, dtype=dtype, mask=torch.from_numpy(m), **kw).verify()


# caps far above the scores: cap tanh(s / cap) is the score itself there
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rules", [dict(), dict(causal=True)])       # whole tiles; tiles that the mask cuts
@pytest.mark.parametrize("cap", [1e3, 1e4, 1e5, 1e6, 1e9, 1e20, 8e37])
def test_caps_above_the_scores(dtype, rules, cap):
    kw = dict(H=2, Nq=256, d=64, dtype=dtype, gain=3.0, **rules)
    c = Narrow(cap=cap, **kw)
    got, ref = c.verify()
    # The same call without a cap, which moves a score of at most 16 by s^3 / 3 cap^2 < 2e-7.  fp32: four roundings of the
    # score, 4 x 16 x 2^-24 in P, twice through the normaliser and twice in P (dP - D): 2^-16.  bf16: a rounding of P, dS or
    # the result may fall to the other side.
    if cap >= 1e5:
        want = Narrow(**kw).run(True)
        for n in ("o", "dq", "dk", "dv"):
            x, y = got[n], want[n].double().cpu().numpy()
            assert np.linalg.norm(x - y) <= (2.0 ** -8 if dtype == BF else 2.0 ** -16) * np.linalg.norm(y), n


# a large cap with a few scores near it, of either sign, among small ones: each score is capped by itself
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("bias", [dict(), dict(slopes=True, buckets=8, distance=30)])
@pytest.mark.parametrize("cap,rules", [(1e4, dict()), (1e5, dict()), (1e5, dict(causal=True))])
def test_large_and_small_scores_under_one_cap(dtype, bias, cap, rules):
    c = Narrow(H=2, Nq=256, d=64, dtype=dtype, cap=cap, **bias, **rules)
    c.k[:, :, ::37] = 0                               # columns with a score of 0 for every row,
    c.k[:, :, 1::37] *= 0
    c.k[:, :, 1::37, 0] = -cap * 8                    # and of about -cap q_0: far below the others or far above
    c.q[:, :, :, 0] = c.q[:, :, :, 0].abs() + 0.25
    c.verify()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cap", [1e-30, 1e-5, 0.3, 60.0])
def test_caps_below_the_scores(dtype, cap):
    Narrow(H=2, Nq=200, d=64, dtype=dtype, cap=cap, scale=3.0 if cap > 1 else 0.125).verify()


# positions far behind the keys: with a slope rows farther from a visible key than fp32 counts (2^24) are refused
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Nq,Nk", [(150, 200), (2, 700)])            # whole tiles, few queries
def test_far_positions_with_slopes(dtype, Nq, Nk):
    lim = 1 << 24
    starts = [1 << 26, lim - Nq + 1, -lim + Nk - 1, 7, 1 << 28]      # beyond, the farthest (both ways), near, beyond
    kw = dict(B=5, H=2, Nq=Nq, Nk=Nk, d=64, dtype=dtype, q_start=starts, kv_len=[Nk, Nk, Nk, Nk, 0], q_len=[Nq] * 5)
    c = Narrow(slopes=True, **kw)
    c.slopes = torch.tensor([2.0 ** -18, 0.0])
    q, k, v, do = (c.gpu(x) for x in (c.q, c.k, c.v, c.do))
    st, sp, skw = torch.zeros(1, dtype=torch.int32, device="cuda"), c.spans(), c.score_kw()
    o, lse = cba.score_attn_fwd(q, k, v, sp, return_lse=True, status=st, **skw)
    grads = cba.score_attn_bwd(do, q, k, v, o, lse, sp, **skw)
    assert st.item() == -2                                           # unsupported
    assert o[0, 0].isnan().all() and lse[0, 0].isnan().all() and grads[0][0, 0].isnan().all()
    assert grads[1][0, 0].isnan().all() and grads[2][0, 0].isnan().all()
    # a head without a slope, the other batch entries and rows that see nothing are as ever
    ref = c.reference(True)
    got = {n: x.double().cpu().numpy() for n, x in zip(("o", "lse", "dq", "dk", "dv"), (o, lse, *grads))}
    for n in got:
        got[n][0, 0] = ref[n][0, 0]
    assert c.faults(got, ref) == []
    # learned buckets clip their offsets: no limit
    Narrow(buckets=8, distance=30, **kw).verify()


# a bucket with the type's lowest value, or -inf, hides its keys; a row that sees nothing else is empty
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kw", [dict(), dict(slopes=True, cap=3.0)])
@pytest.mark.parametrize("low", ["lowest", "-inf"])
@pytest.mark.parametrize("Nq,Nk", [(300, 310), (3, 500)])
def test_lowest_table_values_hide_keys(dtype, kw, low, Nq, Nk):
    c = Narrow(B=2, H=2, Nq=Nq, Nk=Nk, d=64, dtype=dtype, buckets=8, distance=60, bidirectional=False, causal=True,
               q_start=[-2, Nk - Nq], **kw)
    R = len(c.buckets) // 2
    c.buckets[R + 1:] = 7                       # keys after the query: hidden by the table instead of by the rule
    c.buckets[:R + 1] = c.buckets[:R + 1].clamp(max=6)
    c.table[:, 7] = torch.finfo(dtype).min if low == "lowest" else float("-inf")
    q, k, v, do = (c.gpu(x) for x in (c.q, c.k, c.v, c.do))
    sp, skw = cba.attn_spans(2, Nq, Nk, q_start=[-2, Nk - Nq]), c.score_kw()
    o, lse = cba.score_attn_fwd(q, k, v, sp, return_lse=True, **skw)
    grads = cba.score_attn_bwd(do, q, k, v, o, lse, sp, **skw)
    c.table[:, 7] = 0                           # (no pair of the reference has bucket 7)
    ref = c.reference(True)
    got = {n: x.double().cpu().numpy() for n, x in zip(("o", "lse", "dq", "dk", "dv", "dtable"), (o, lse, *grads))}
    assert c.faults(got, ref) == [] and (got["lse"][0, :, :2] == -np.inf).all()


def test_map_offset_beyond_int_is_refused():
    q = torch.zeros(1, 2, 130, 64, dtype=BF, device="cuda")
    mask = torch.ones(4, 2, 2, dtype=torch.uint8, device="cuda")
    for off in (1 << 32, (1 << 32) + 2, -(1 << 32)):
        with pytest.raises(cba.CalibattError, match="map_offset"):
            cba.score_attn_fwd(q, q, q, cba.attn_spans(1, 130, 130), mask=mask, map_offset=off)


# steep slopes: buckets whose gradient is far below their neighbours' keep their own digits
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kw", [
    dict(H=5, Hkv=1, Nq=108, Nk=759, cap=50.0, buckets=64, distance=79, docs=[[45, 225, 263, 612, 697]], q_start=[434], seed=633140, steep=4),
    dict(H=5, Hkv=1, Nq=108, Nk=759, cap=50.0, buckets=64, distance=79, docs=[[45, 225, 263, 612, 697]], q_start=[434], seed=633140, steep=-1),
    dict(H=2, Nq=200, buckets=8, distance=400, steep=4), dict(H=2, Nq=200, buckets=8, distance=400, steep=-8, causal=True),
    dict(H=4, Nq=300, buckets=16, distance=60, steep=16), dict(H=2, Nq=300, d=128, buckets=32, distance=120, causal=True, steep=8),
])
def test_small_buckets_beside_large_ones(dtype, kw):
    kw = dict(kw)
    steep = kw.pop("steep", 1)
    c = Narrow(dtype=dtype, slopes=True, **kw)
    c.slopes = c.slopes * steep
    c.verify()
