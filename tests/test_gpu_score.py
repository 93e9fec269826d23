"""Score-modified attention on the GPU against the float64 oracle, elementwise
within the bounds that tests/_score_util.py derives."""

import numpy as np
import pytest
import torch

import block_sparse_attention_cross_b200 as cba
from oracle import score as osc
from tests._score_util import Case

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("B,Nq,Nk,rules", [
    (2, 300, 300, dict(causal=True)),
    (3, 257, 511, dict(kv_len=[511, 1, 0], q_start=[254, 0, 3], causal=True)),
    (2, 130, 130, dict(docs=[[0, 5, 5, 100, 128], [1, 2, 60, 61, 130]], causal=True, prefix=[[2, 9, 3, 500], [1, 0, 1, 7]])),
    (2, 130, 140, dict(docs=[[0, 50, 140], [0, 0, 0]], kv_len=[60, 100], q_len=[130, 4])),
    (1, 1, 1, dict()),
])
def test_spans(B, Nq, Nk, rules):
    sp = cba.attn_spans(B, Nq, Nk, **rules)
    vis = osc.spans(B, Nq, Nk, **rules)
    row = sp.row.cpu().numpy()
    for b in range(B):
        for i in range(Nq):
            lo, hi = row[b, i]
            keys = np.flatnonzero(vis[b, i])
            assert (hi - lo) == len(keys) and (len(keys) == 0 or (keys[0] == lo and keys[-1] == hi - 1))
        for t in range(-(-Nq // 128)):
            r = row[b, t * 128:(t + 1) * 128]
            live = r[r[:, 1] > r[:, 0]]
            x = sp.tile[b, t].cpu().numpy()
            assert (x[0], x[1]) == ((live[:, 0].min(), live[:, 1].max()) if len(live) else (0, 0))
            assert x[2] == (Nk if len(live) < len(r) else live[:, 0].max())
            assert x[3] == (0 if len(live) < len(r) else live[:, 1].min())


# lengths around the tile sizes, from one token on
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [1, 2, 63, 127, 128, 129, 300])
def test_lengths(dtype, d, N):
    Case(Nq=N, d=d, dtype=dtype, seed=N).check()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kw", [
    dict(cap=5.0), dict(cap=50.0, gain=8.0), dict(slopes=True), dict(buckets=16, distance=12),
    dict(buckets=32, distance=200), dict(buckets=8, distance=1000, bidirectional=False, causal=True),
    dict(cap=2.0, slopes=True, buckets=6, distance=40, causal=True),
    dict(buckets=256, distance=300, cap=4.0),
])
def test_scores(dtype, kw):
    Case(H=3, Nq=333, dtype=dtype, **kw).check()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kw", [
    dict(causal=True),
    dict(causal=True, prefix=[[40], [300]]),
    dict(docs=[[0, 100, 101, 270], [3, 3, 130, 260]]),
    dict(docs=[[0, 100, 101, 270], [3, 3, 130, 260]], causal=True, prefix=[[1, 1, 64], [5, 100, 2]]),
    dict(kv_len=[270, 5], q_len=[270, 5]),
    dict(kv_len=[0, 129], q_len=[0, 200]),
])
def test_masks(dtype, kw):
    Case(B=2, H=4, Hkv=2, Nq=270, d=64, dtype=dtype, cap=3.0, slopes=True, buckets=12, distance=50, **kw).check()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,Hkv,d", [(4, 1, 128), (6, 2, 64), (5, 5, 128)])
def test_heads_and_layout(dtype, H, Hkv, d):
    Case(B=2, H=H, Hkv=Hkv, Nq=140, d=d, dtype=dtype, layout="bnhd", causal=True, cap=6.0, buckets=10,
         distance=30).check()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kw", [dict(), dict(cap=4.0, slopes=True, buckets=16, distance=70), dict(causal=True)])
def test_calibrated_mask(dtype, kw):
    rng = np.random.default_rng(7)
    m = (rng.random((2, 4, 4)) < 0.5).astype(np.uint8)
    m[1, 2] = 0            # a query tile without any kept block
    m[0, 0] = [0, 0, 0, 1]  # with the causal rule: kept, but not visible
    Case(H=2, Nq=450, d=128, dtype=dtype, mask=torch.from_numpy(m), **kw).check()


# single tokens and a few against long and ragged key axes
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Nq,Nk,H,Hkv,d", [(1, 1, 2, 2, 64), (1, 700, 8, 2, 128), (3, 2500, 4, 4, 64), (5, 1111, 16, 2, 128),
                                           (17, 4000, 10, 1, 64), (130, 1500, 4, 2, 128)])
@pytest.mark.parametrize("kw", [dict(), dict(cap=5.0, slopes=True, buckets=16, distance=600)])
def test_few_queries(dtype, Nq, Nk, H, Hkv, d, kw):
    lens = [Nk, max(1, Nk // 3), 1]
    Case(B=3, H=H, Hkv=Hkv, Nq=Nq, Nk=Nk, d=d, dtype=dtype, causal=True, kv_len=lens,
         q_start=[max(0, n - Nq) for n in lens], q_len=[min(n, Nq) for n in lens], **kw).check(train=Nk < 1200)


# queries and keys of unrelated lengths (no causal rule)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_cross_lengths(dtype):
    Case(B=2, H=2, Nq=400, Nk=77, d=64, dtype=dtype, kv_len=[77, 30], cap=8.0).check()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_masked_nan_and_inf_do_not_matter(dtype):
    # garbage behind the lengths (whole keys and queries) and in other documents
    c = Case(B=2, H=2, Hkv=1, Nq=300, d=64, dtype=dtype, cap=5.0, buckets=8, distance=20,
             docs=[[0, 90, 200, 300], [0, 150, 160, 300]], kv_len=[260, 300], q_len=[260, 300])
    want = c.run(True)
    for x, val in ((c.k, float("nan")), (c.v, float("inf")), (c.q, float("nan")), (c.do, float("-inf"))):
        x[0, :, 260:] = val
    got = c.run(True)
    for name in want:
        assert torch.equal(want[name], got[name]), name
    # document 1 of batch entry 0 becomes NaN, the others keep their results
    c.v[0, :, 120] = float("nan")
    c.k[0, :, 130] = float("nan")
    c.q[0, :, 140] = float("nan")
    c.do[0, :, 150] = float("nan")
    got = c.run(True)
    for name in ("o", "dq", "dk", "dv"):
        assert torch.equal(want[name][0, :, :90], got[name][0, :, :90]), name
        assert torch.equal(want[name][0, :, 200:], got[name][0, :, 200:]), name
        assert torch.equal(want[name][1], got[name][1]), name
    assert got["o"][0, :, 90:200].isnan().all()
    assert got["dv"][0, :, 90:200].isnan().all() and got["dk"][0, :, 90:200].isnan().all()


def test_forward_rows_of_full_tiles_see_nan():
    c = Case(H=1, Nq=128, d=64)
    c.v[0, 0, 5, 3] = float("nan")
    assert c.run(False)["o"][0, 0, :, 3].isnan().all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_extreme_scores(dtype):
    # one dominant key a row, and differences far beyond the range of exp
    c = Case(H=1, Nq=260, d=64, dtype=dtype, scale=4.0, gain=6.0)
    c.check()
    c = Case(H=1, Nq=260, d=64, dtype=dtype, scale=4.0, gain=6.0, cap=100.0)
    c.check()


def test_corrupt_bucket_map_is_reported():
    for dtype in (BF, F32):
        c = Case(H=1, Nq=40, dtype=dtype, buckets=8, distance=20)
        kw = c.score_kw()
        kw["buckets"][20] = 8
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        cba.score_attn_fwd(c.gpu(c.q), c.gpu(c.k), c.gpu(c.v), c.spans(), status=st, **kw)
        assert st.item() == -5


def test_deterministic_and_graph_replay():
    c = Case(B=2, H=4, Hkv=2, Nq=500, d=128, cap=5.0, slopes=True, buckets=32, distance=100, causal=True)
    first = c.run(True)
    kw = c.score_kw()
    q, k, v, do = (c.gpu(x) for x in (c.q, c.k, c.v, c.do))
    sp = c.spans()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        o, lse = cba.score_attn_fwd(q, k, v, sp, return_lse=True, **kw)
        grads = cba.score_attn_bwd(do, q, k, v, o, lse, sp, **kw)
    g2 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g2):
        o2, _ = cba.score_attn_fwd(q[:1], k[:1], v[:1], cba.attn_spans(1, 500, 500, causal=True), return_lse=True, **kw)
    for _ in range(2):
        g.replay()
        g2.replay()
        torch.cuda.synchronize()
        for name, x in zip(("o", "lse", "dq", "dk", "dv", "dtable"), (o, lse, *grads)):
            assert torch.equal(x, first[name]), name
        assert torch.equal(o2, first["o"][:1])


@pytest.mark.parametrize("kw", [dict(cap=50.0, prefix=[1000]), dict(prefix=[1000]),
                                dict(cap=50.0, docs=[[0, 700, 1500, 2046]], prefix=[[650, 500, 546]])])
def test_repeated_backward_is_bit_equal(kw):
    # Rows before the prefix's end see keys after them (one bucket, summed fast) and near the diagonal many buckets
    # (summed slowly): the warps of a tile run apart, and no tile may be used before the slowest has stored its part.
    N = 2046
    c = Case(H=16, Hkv=4, Nq=N, d=128, buckets=64, distance=8192, bidirectional=False, causal=True, **kw)
    skw, sp = c.score_kw(), c.spans()
    q, k, v, do = (c.gpu(x) for x in (c.q, c.k, c.v, c.do))
    o, lse = cba.score_attn_fwd(q, k, v, sp, return_lse=True, **skw)
    first = cba.score_attn_bwd(do, q, k, v, o, lse, sp, **skw)
    assert all(torch.isfinite(x).all() for x in first)
    for _ in range(20):
        again = cba.score_attn_bwd(do, q, k, v, o, lse, sp, **skw)
        for name, x, y in zip(("dq", "dk", "dv", "dtable"), first, again):
            assert torch.equal(x, y), name


def test_caller_buffers_and_refusals():
    c = Case(B=1, H=2, Nq=33, d=64, buckets=4, distance=3)
    q, k, v = (c.gpu(x) for x in (c.q, c.k, c.v))
    sp, kw = c.spans(), c.score_kw()
    out, lse = torch.full_like(q, 7), torch.full((1, 2, 33), 7.0, device="cuda")
    r = cba.score_attn_fwd(q, k, v, sp, out=out, lse=lse, **kw)
    assert r.data_ptr() == out.data_ptr() and not (lse == 7).any()
    for bad in (dict(cap=-1.0), dict(cap=float("nan")), dict(scale=0.0), dict(scale=float("inf"))):
        with pytest.raises(cba.CalibattError):
            cba.score_attn_fwd(q, k, v, sp, **{**kw, **bad})
    for bad in (dict(table=None), dict(table=kw["table"].float()), dict(table=kw["table"][:1]),
                dict(buckets=kw["buckets"].long()), dict(buckets=kw["buckets"][:-1]), dict(slopes=torch.ones(3, device="cuda")),
                dict(mask=torch.ones(2, 2, 1, dtype=torch.uint8, device="cuda")),
                dict(out=torch.empty(1, 2, 33, 32, device="cuda", dtype=BF))):
        with pytest.raises(ValueError):
            cba.score_attn_fwd(q, k, v, sp, **{**kw, **bad})
    with pytest.raises(cba.CalibattError, match="map_offset"):
        cba.score_attn_fwd(q, k, v, sp, mask=torch.ones(2, 1, 1, dtype=torch.uint8, device="cuda"), map_offset=1)
    with pytest.raises(ValueError, match="strides"):
        cba.score_attn_fwd(q, k[:, :1].expand(1, 2, 33, 64), v, sp)
    with pytest.raises(ValueError, match="strides"):
        cba.score_attn_fwd(torch.empty(1, 2, 33, 65, device="cuda", dtype=BF)[..., :64], k, v, sp)
    with pytest.raises(cba.CalibattError, match="aligned"):
        buf = torch.empty(2 * 33 * 64 + 8, device="cuda", dtype=BF)
        cba.score_attn_fwd(buf[1:1 + 2 * 33 * 64].view(1, 2, 33, 64), k, v, sp)
    with pytest.raises(cba.CalibattError, match="overlap"):
        cba.score_attn_fwd(q, k, v, sp, out=torch.empty(64 * 34, device="cuda", dtype=BF).as_strided((1, 2, 33, 64), (0, 64, 64, 1)))
    with pytest.raises(cba.CalibattError, match="d must be"):
        x = torch.zeros(1, 2, 33, 96, device="cuda", dtype=BF)
        cba.score_attn_fwd(x, x, x, sp)
    with pytest.raises(ValueError, match="lse"):
        cba.score_attn_bwd(q, q, k, v, out, None, sp)


def test_lse_is_optional_and_streams_and_sizes_mix():
    # without an LSE, on another stream, one call after another of other sizes: the same bits
    side = torch.cuda.Stream()
    for kw in (dict(Nq=300, H=4, Hkv=2, cap=5.0), dict(Nq=2, Nk=900, H=8, Hkv=2, d=128, causal=True, q_start=[898], buckets=8, distance=90),
               dict(Nq=70, H=2, slopes=True, dtype=F32)):
        c = Case(**kw)
        want = c.run(False)["o"]
        q, k, v = (c.gpu(x) for x in (c.q, c.k, c.v))
        sp, skw = c.spans(), c.score_kw()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            o = cba.score_attn_fwd(q, k, v, sp, **skw)
        side.synchronize()
        assert torch.equal(o, want)


# caps far from the scores on either side (the cap's polynomial is left there)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cap,scale", [(1e-5, 0.125), (1e6, 0.125), (1e5, 4000.0), (60.0, 3.0)])
def test_caps_of_every_size(dtype, cap, scale):
    Case(H=1, Nq=150, d=64, dtype=dtype, cap=cap, scale=scale, gain=1e-2 if cap > 1e4 and scale > 1 else 1.0).check()


# values far from 1 on either side, every score at the cap's negative end for some rows
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("size", [1e9, 1e-6])
def test_sizes_of_values_under_a_cap(dtype, size):
    c = Case(H=2, Nq=200, d=64, dtype=dtype, cap=55.0, scale=8.0, gain=4.0)
    c.v = (c.v.float() * size).to(dtype)
    c.k[0, 0] = c.k[0, 0, :1]
    c.q[0, 0, 50:120] = -8 * c.k[0, 0, 0]
    c.check(train=False)


def test_integers_of_any_width_and_place():
    want = cba.attn_spans(2, 40, 50, causal=True, kv_len=[50, 7], q_start=[10, 0], prefix=[3, 60])
    got = cba.attn_spans(2, 40, 50, causal=True, kv_len=torch.tensor([1 << 40, 7], device="cuda"),
                         q_start=torch.tensor([10, 0], dtype=torch.int16), prefix=np.array([[3], [60]]))
    assert torch.equal(want.row, got.row) and torch.equal(want.tile, got.tile)


def test_calls_on_two_streams_at_once():
    cases = [Case(B=2, H=4, Hkv=2, Nq=700, d=128, cap=9.0, buckets=16, distance=60, causal=True),
             Case(B=1, H=6, Hkv=2, Nq=3, Nk=3000, slopes=True)]
    want = [c.run(c.sizes[3] > 3) for c in cases]
    data = [([c.gpu(x) for x in (c.q, c.k, c.v, c.do)], c.spans(), c.score_kw()) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, st in enumerate(streams):
            (q, k, v, do), sp, kw = data[i]
            with torch.cuda.stream(st):
                o, lse = cba.score_attn_fwd(q, k, v, sp, return_lse=True, **kw)
                got[i].append([o, lse])
                if i == 0:
                    got[i][-1] += cba.score_attn_bwd(do, q, k, v, o, lse, sp, **kw)
    torch.cuda.synchronize()
    for i in range(2):
        for run in got[i]:
            for name, x in zip(("o", "lse", "dq", "dk", "dv", "dtable"), run):
                assert torch.equal(x, want[i][name]), name


def test_map_offset_picks_the_heads_masks():
    rng = np.random.default_rng(3)
    maps = torch.from_numpy((rng.random((7, 3, 3)) < 0.6).astype(np.uint8))
    c = Case(H=2, Nq=300, mask=maps[4:6].contiguous(), cap=7.0)
    want = c.run(True)
    q, k, v, do = (c.gpu(x) for x in (c.q, c.k, c.v, c.do))
    sp, kw = c.spans(), {**c.score_kw(), "mask": maps.cuda(), "map_offset": 4}
    o, lse = cba.score_attn_fwd(q, k, v, sp, return_lse=True, **kw)
    g = cba.score_attn_bwd(do, q, k, v, o, lse, sp, **kw)
    for name, x in zip(("o", "lse", "dq", "dk", "dv"), (o, lse, *g)):
        assert torch.equal(x, want[name]), name


# a cache of 2^31 elements a tensor: all keys and values 0 but the last 40 of the last head
def test_offsets_beyond_32_bits():
    H, Nk, d, tail = 8, (1 << 21) + 77, 128, 40
    g = torch.Generator().manual_seed(1)
    k = torch.zeros(1, H, Nk, d, dtype=BF, device="cuda")
    v = torch.zeros_like(k)
    kt, vt = torch.randn(tail, d, generator=g).to(BF), torch.randn(tail, d, generator=g).to(BF)
    k[0, -1, -tail:], v[0, -1, -tail:] = kt.cuda(), vt.cuda()
    q = (torch.randn(1, H, 2, d, generator=g) * 4).to(BF)
    o, lse = cba.score_attn_fwd(q.cuda(), k, v, cba.attn_spans(1, 2, Nk), scale=0.25, return_lse=True)
    e = torch.exp(0.25 * q[0, -1].double() @ kt.double().T)          # every other key: exp(0) and a value of 0
    norm = e.sum(1) + (Nk - tail)
    want = (e @ vt.double()) / norm[:, None]
    # probabilities, normaliser and result rounded to bf16 (2^-8 each); the fp32 sum of 2^21 terms of 1 in
    # 128 x 16384 partial sums is off by at most 2^-24 x 2^14
    bound = 4 * 2.0 ** -8 * ((e @ vt.double().abs()) / norm[:, None])
    assert ((o[0, -1].double().cpu() - want).abs() <= bound).all()
    assert torch.allclose(lse[0, -1].double().cpu(), norm.log(), rtol=0, atol=2.0 ** -9)
    assert (o[0, :-1] == 0).all() and torch.allclose(lse[0, :-1].double().cpu(), torch.tensor(float(Nk)).double().log(), rtol=0,
                                                     atol=2.0 ** -9)


# a row's bits do not depend on other rows, heads or batch entries
def test_rows_stand_alone():
    c = Case(B=2, H=4, Hkv=2, Nq=260, d=128, cap=20.0, buckets=8, distance=40, causal=True)
    want = c.run(True)
    c.q[1, 3, 100:] *= 50      # beyond the polynomial's range
    c.k[1, 1, 230:] *= 30
    got = c.run(True)
    for name in ("o", "dq"):
        assert torch.equal(want[name][0], got[name][0]), name
        assert torch.equal(want[name][1, :2], got[name][1, :2]), name
        assert torch.equal(want[name][1, 3, :100], got[name][1, 3, :100]), name


def test_fused_projection_views():
    # q, k, v as slices of one [B, N, 3, H, d] projection
    g = torch.Generator().manual_seed(5)
    x = torch.randn(2, 200, 3, 2, 64, generator=g).to(BF)
    c = Case(B=2, H=2, Nq=200, d=64, cap=4.0, causal=True)
    c.q, c.k, c.v = (x[:, :, i].transpose(1, 2) for i in range(3))
    dev = x.cuda()
    kw, sp = c.score_kw(), c.spans()
    o, lse = cba.score_attn_fwd(*(dev[:, :, i].transpose(1, 2) for i in range(3)), sp, return_lse=True, **kw)
    grads = cba.score_attn_bwd(c.do.cuda(), *(dev[:, :, i].transpose(1, 2) for i in range(3)), o, lse, sp, **kw)
    ref = c.reference(True)
    b = c.bounds(ref, True)
    for name, y in zip(("o", "lse", "dq", "dk", "dv"), (o, lse, *grads)):
        assert (np.abs(y.double().cpu().numpy() - ref[name]) <= b[name]).all(), name


def test_calibrate_then_train_under_the_mask():
    # the masks that calibrate() returns, used as they are: forward and gradients
    H, N, Np, d = 2, 500, 512, 64
    g = torch.Generator().manual_seed(9)
    x = [torch.randn(H, Np, d, generator=g).to(BF).cuda() for _ in range(2)]
    mask, _, _ = cba.calibrate([x[0]], [x[1]], N, select_param=0.5, rho=0.5)
    c = Case(H=H, Nq=N, d=d, mask=mask.cpu(), cap=6.0, seed=3)
    got, _ = c.check()
    # without a cap the forward agrees with the block-sparse forward on the same inputs
    c = Case(H=H, Nq=N, d=d, mask=mask.cpu(), seed=3)
    got = c.run(False)
    pad = lambda t: torch.nn.functional.pad(t, (0, 0, 0, Np - N)).cuda()   # noqa: E731
    o, lse = cba.sparse_attn_fwd(pad(c.q), pad(c.k), pad(c.v), cba.compile(mask), N, scale=c.scale, return_lse=True)
    ref = c.reference(False)
    bound = c.bounds(ref, False)
    diff = np.abs(o[:, :, :N].double().cpu().numpy() - got["o"].double().cpu().numpy())
    assert (diff <= 2 * bound["o"]).all()
