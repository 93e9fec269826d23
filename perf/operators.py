"""What is measured of the score-modified attention operators.

Three operators over one definition.  Query row i of batch entry b stands at
key position p = q_start[b] + i and sees the keys j of one interval
[lo, hi) (documents, a causal or prefix rule, lengths; empty for padding
rows), further restricted to the kept 128 x 128 blocks of a calibrated mask
where one is given:

    s_ij  = scale q_i.k_j;   c_ij = cap tanh(s_ij / cap)   (c = s without a cap)
    z_ij  = c_ij - slope_h |j - p| + table[h, bucket(j - p)]
    O_i   = sum_j softmax_j(z_ij) v_j,   LSE_i = ln sum_j exp z_ij

* forward       kind "fwd": prompts and whole clips, and single tokens (few
                query rows against a long key axis);
* training      kind "train": forward, then dQ, dK, dV of a given dO;
* learned bias  either kind with "buckets" > 0: the table enters the scores,
                and training also returns its gradient.

``own`` selects the framework's kernels; otherwise the plain torch form runs.
"""

import math
import random

import numpy as np
import torch

own = False

BLOCK = 128
NEG = float("-inf")
_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}

_DEFAULTS = dict(kind="fwd", B=1, H=8, Hkv=8, Nq=128, Nk=128, d=128, dtype="bf16", cap=0.0, slopes=False, buckets=0,
                 distance=128, causal=False, docs=0, prefix=0, padded=False, kept=1.0, layout="bhnd")


def _case(name, **kw):
    c = dict(_DEFAULTS)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one new token of one sequence: nothing but latency
        _case("token_small", H=8, Hkv=8, Nq=1, Nk=513, d=64, cap=30.0),
        # a serving step: one token of 32 sequences of different lengths, five query heads to a key head
        _case("token_batch", B=32, H=40, Hkv=8, Nq=1, Nk=8191, cap=50.0, slopes=True, padded=True),
        # four tokens against the 720p clip's keys: little parallelism but the key axis
        _case("token_long_bias", H=24, Hkv=24, Nq=4, Nk=75600, buckets=32, distance=4096, causal=True),
        # a text encoder's batch, padded to its longest prompt
        _case("text_bias", B=4, H=16, Hkv=16, Nq=512, Nk=512, d=64, buckets=32, distance=128, padded=True),
        # packed clips of different lengths, [B, N, H, d] activations seen as [B, H, N, d]
        _case("packed_clips", B=2, H=40, Hkv=40, Nq=7801, Nk=7801, docs=9, slopes=True, layout="bnhd"),
        # a conditioning prefix seen by all, then causal generation
        _case("prefix_capped", H=24, Hkv=8, Nq=11233, Nk=11233, cap=30.0, causal=True, prefix=1560),
        # the 480p clip (8 heads) under a calibrated 25% mask with capped scores
        _case("clip480_capped_mask", H=8, Hkv=8, Nq=32760, Nk=32760, cap=50.0, kept=0.25),
        # exact-check type
        _case("fp32_capped", B=1, H=4, Hkv=4, Nq=1001, Nk=1001, d=64, dtype="fp32", cap=20.0, slopes=True, causal=True),
        # training on packed clips
        _case("train_packed_capped", kind="train", H=16, Hkv=16, Nq=6145, Nk=6145, cap=50.0, slopes=True, causal=True,
              docs=5),
        # training an encoder with a learned bias
        _case("train_bias", kind="train", B=2, H=12, Hkv=12, Nq=3900, Nk=3900, d=64, buckets=32, distance=128),
        # the same with a prefix, shared key heads and far distances; the largest backward
        _case("train_bias_prefix", kind="train", H=16, Hkv=4, Nq=8190, Nk=8190, buckets=64, distance=8192, causal=True,
              prefix=1000, cap=50.0),
        # a small training step in the exact-check type
        _case("train_fp32_bias", kind="train", B=2, H=2, Hkv=2, Nq=257, Nk=257, d=64, dtype="fp32", buckets=16,
              distance=64, padded=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    H = Hkv * rng.choice([1, 1, 2, 5])
    feat = dict(cap=rng.choice([0.0, 20.0, 50.0]), slopes=rng.random() < 0.4,
                buckets=rng.choice([0, 0, 16, 32, 64]), distance=_log_int(rng, 33, 8192),
                layout=rng.choice(["bhnd", "bnhd"]))
    what = rng.choice(["token", "prompt", "prompt", "train", "train", "fp32"])
    if what == "token":
        return _case("", B=_log_int(rng, 1, 24), H=H, Hkv=Hkv, Nq=rng.choice([1, 1, 2, 5]), Nk=_log_int(rng, 1, 30000),
                     d=d, padded=rng.random() < 0.5, causal=rng.random() < 0.5, **feat)
    shape = rng.choice(["whole", "docs", "prefix", "padded"])
    kw = dict(docs=rng.randint(2, 9) if shape == "docs" else 0, padded=shape == "padded",
              causal=shape == "prefix" or rng.random() < 0.4)
    if what == "fp32":
        n = _log_int(rng, 1, 700)
        kw["prefix"] = n // 4 if shape == "prefix" else 0
        return _case("", kind=rng.choice(["fwd", "train"]), B=rng.randint(1, 2), H=H, Hkv=Hkv, Nq=n, Nk=n, d=d,
                     dtype="fp32", **kw, **feat)
    if what == "train":
        n = _log_int(rng, 100, 5000)
        kw["prefix"] = n // 4 if shape == "prefix" else 0
        return _case("", kind="train", B=rng.randint(1, 2), H=H, Hkv=Hkv, Nq=n, Nk=n, d=d, **kw, **feat)
    n = _log_int(rng, 60, 12000)
    kw["prefix"] = n // 4 if shape == "prefix" else 0
    kept = rng.choice([0.3, 1.0]) if shape == "whole" and n > 2000 else 1.0
    return _case("", B=rng.randint(1, 2), H=H, Hkv=Hkv, Nq=n, Nk=n, d=d, kept=kept, **kw, **feat)


# ---- geometry: a function of the case alone --------------------------------


def _bounds(case):
    """Document bounds [B][docs + 1], key lengths [B], query lengths [B], query starts [B], prefix lengths [B][docs or 1]."""
    B, Nq, Nk = case["B"], case["Nq"], case["Nk"]
    rng = random.Random(1000003 * Nk + 101 * Nq + B)
    docs = None
    if case["docs"]:
        docs = []
        for _ in range(B):
            cuts = sorted(rng.randint(0, Nk) for _ in range(case["docs"] - 1))
            docs.append([0] + cuts + [Nk - rng.randint(0, Nk // 50)])
    kv_len = [Nk] * B
    if case["padded"]:
        kv_len = [max(1, Nk - int(Nk * 0.7 * rng.random())) for _ in range(B)]
        kv_len[0] = Nk
    if Nq == Nk:
        q_len, q_start = list(kv_len), [0] * B
    else:  # the last Nq tokens of every sequence
        q_len, q_start = [min(Nq, n) for n in kv_len], [max(0, n - Nq) for n in kv_len]
    prefix = [[case["prefix"]] * max(1, case["docs"]) for _ in range(B)]
    return docs, kv_len, q_len, q_start, prefix


def _intervals(case):
    """Visible interval [lo, hi) of every row, int64 numpy [B, Nq] each."""
    docs, kv_len, q_len, q_start, prefix = _bounds(case)
    B, Nq = case["B"], case["Nq"]
    lo = np.zeros((B, Nq), np.int64)
    hi = np.zeros((B, Nq), np.int64)
    for b in range(B):
        for i in range(min(Nq, q_len[b])):
            p = q_start[b] + i
            s, e, pre = 0, kv_len[b], prefix[b][0]
            if docs is not None:
                m = 0
                while m < case["docs"] and not (docs[b][m] <= p < docs[b][m + 1]):
                    m += 1
                if m == case["docs"]:
                    continue
                s, e, pre = docs[b][m], min(docs[b][m + 1], kv_len[b]), prefix[b][m]
            if case["causal"]:
                e = min(e, max(p + 1, s + pre))
            lo[b, i], hi[b, i] = s, max(s, e)
    return lo, hi


def _kept_blocks(case):
    """Calibrated mask uint8 [H, query blocks, key blocks] (diagonal kept) or None."""
    if case["kept"] >= 1.0:
        return None
    nq, nk = -(-case["Nq"] // BLOCK), -(-case["Nk"] // BLOCK)
    rng = np.random.default_rng(case["Nk"] * 7 + case["H"])
    m = (rng.random((case["H"], nq, nk)) < case["kept"]).astype(np.uint8)
    for i in range(min(nq, nk)):
        m[:, i, i] = 1
    return m


def _bucket_map(n, distance, causal):
    """Bucket of every clipped offset -distance .. distance: exact near zero, logarithmic out to the distance."""
    half = n if causal else n // 2
    exact = half // 2
    out = np.zeros(2 * distance + 1, np.int32)
    for k, off in enumerate(range(-distance, distance + 1)):
        a = abs(off)
        if a < exact:
            b = a
        else:
            b = exact + int((half - exact) * math.log(a / exact) / math.log(max(distance, exact + 1) / exact))
        b = min(b, half - 1)
        if causal:
            b = 0 if off > 0 else b
        elif off > 0:
            b += half
        out[k] = b
    return out


def work(case):
    lo, hi = _intervals(case)
    B, H, Hkv, Nq, Nk, d = (case[k] for k in ("B", "H", "Hkv", "Nq", "Nk", "d"))
    esz = 2 if case["dtype"] == "bf16" else 4
    m = _kept_blocks(case)
    if m is None:
        pairs = float((hi - lo).sum()) * H
    else:
        pairs = 0.0
        size = np.minimum(BLOCK, Nk - BLOCK * np.arange(m.shape[2]))
        rows = np.minimum(BLOCK, Nq - BLOCK * np.arange(m.shape[1]))
        pairs = B * float(np.einsum("hqk,q,k->", m.astype(np.float64), rows, size))
    keys = float(np.maximum(hi.max(1) - lo.min(1), 0).sum())     # keys that some row can see
    q_el, kv_el = float(B * H * Nq * d), keys * Hkv * d
    nbytes = esz * (2 * q_el + 2 * kv_el) + 4.0 * B * H * Nq
    flops = 4.0 * d * pairs
    if case["kind"] == "train":
        nbytes += esz * (2 * q_el + 2 * B * Hkv * Nk * d)        # dO in, dQ, dK, dV out
        flops += 10.0 * d * pairs
    return {"bytes": nbytes, "flops": flops}


# ---- inputs -----------------------------------------------------------------


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = _DT[case["dtype"]]
    B, H, Hkv, Nq, Nk, d = (case[k] for k in ("B", "H", "Hkv", "Nq", "Nk", "d"))

    def acts(h, n, gain=1.0):
        if case["layout"] == "bnhd":
            return (torch.randn(B, n, h, d, device="cuda", generator=g) * gain).to(dt).transpose(1, 2)
        return (torch.randn(B, h, n, d, device="cuda", generator=g) * gain).to(dt)

    docs, kv_len, q_len, q_start, prefix = _bounds(case)

    def ints(x):
        return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")

    st = {"case": case, "q": acts(H, Nq, 2.0), "k": acts(Hkv, Nk), "v": acts(Hkv, Nk), "scale": 1.0 / math.sqrt(d),
          "docs": ints(docs), "kv_len": ints(kv_len), "q_len": ints(q_len), "q_start": ints(q_start),
          "prefix": ints(prefix) if case["prefix"] else None, "slopes": None, "table": None, "buckets": None,
          "do": None, "mask": None}
    if case["slopes"]:
        st["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], device="cuda")
    if case["buckets"]:
        st["table"] = torch.randn(H, case["buckets"], device="cuda", generator=g).to(dt)
        st["buckets"] = torch.from_numpy(_bucket_map(case["buckets"], case["distance"], case["causal"])).cuda()
    if case["kind"] == "train":
        st["do"] = acts(H, Nq)
    m = _kept_blocks(case)
    if m is not None:
        st["mask"] = torch.from_numpy(m).cuda()
    if own:
        import block_sparse_attention_cross_b200 as cba
        st["spans"] = cba.attn_spans(B, Nq, Nk, causal=case["causal"], docs=st["docs"], prefix=st["prefix"],
                                     kv_len=st["kv_len"], q_len=st["q_len"], q_start=st["q_start"], device="cuda")
    return st


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(st):
    import block_sparse_attention_cross_b200 as cba
    kw = dict(scale=st["scale"], cap=st["case"]["cap"], slopes=st["slopes"], table=st["table"], buckets=st["buckets"],
              mask=st["mask"])
    o, lse = cba.score_attn_fwd(st["q"], st["k"], st["v"], st["spans"], return_lse=True, **kw)
    if st["do"] is None:
        return {"o": o, "lse": lse}
    grads = cba.score_attn_bwd(st["do"], st["q"], st["k"], st["v"], o, lse, st["spans"], **kw)
    out = {"o": o, "lse": lse, "dq": grads[0], "dk": grads[1], "dv": grads[2]}
    if st["table"] is not None:
        out["dtable"] = grads[3]
    return out


# ---- the plain form -----------------------------------------------------------


def _visible(st, b):
    """bool [Nq, Nk] of batch entry b, from the lengths, documents and rules."""
    case = st["case"]
    Nq, Nk = case["Nq"], case["Nk"]
    i = torch.arange(Nq, device="cuda")[:, None]
    j = torch.arange(Nk, device="cuda")[None, :]
    p = i + st["q_start"][b]
    vis = (i < st["q_len"][b]) & (j < st["kv_len"][b])
    start = torch.zeros_like(p)
    pre = st["prefix"][b][0] if st["prefix"] is not None else 0
    if st["docs"] is not None:
        bounds = st["docs"][b]
        dq = torch.searchsorted(bounds, p[:, 0].to(torch.int32), right=True) - 1
        dk = torch.searchsorted(bounds, j[0].to(torch.int32), right=True) - 1
        last = bounds.numel() - 1
        vis = vis & (dq[:, None] == dk[None, :]) & (dq[:, None] >= 0) & (dq[:, None] < last)
        at = dq.clamp(0, last - 1)
        start = bounds[at][:, None]
        if st["prefix"] is not None:
            pre = st["prefix"][b][at][:, None]
    if case["causal"]:
        vis = vis & ((j <= p) | (j < start + pre))
    return vis


def _offsets(st, b):
    case = st["case"]
    i = torch.arange(case["Nq"], device="cuda")[:, None]
    j = torch.arange(case["Nk"], device="cuda")[None, :]
    return j - (i + st["q_start"][b])


def _run_plain(st):
    case = st["case"]
    B, H, Hkv, Nq, Nk, d = (case[k] for k in ("B", "H", "Hkv", "Nq", "Nk", "d"))
    G = H // Hkv
    q, k, v, do, cap = st["q"], st["k"], st["v"], st["do"], case["cap"]
    o = torch.empty_like(q)
    lse = torch.empty(B, H, Nq, device="cuda")
    train = do is not None
    if train:
        dq, dk32, dv32 = torch.empty_like(q), torch.zeros(k.shape, device="cuda"), torch.zeros(v.shape, device="cuda")
        if st["table"] is not None:
            dtable = torch.zeros(st["table"].shape, device="cuda", dtype=torch.float64)
    chunk = max(1, min(G, (1 << 28) // (Nq * Nk)))
    for b in range(B):
        vis = _visible(st, b)
        off = _offsets(st, b) if (st["slopes"] is not None or st["table"] is not None) else None
        if st["table"] is not None:
            R = (st["buckets"].numel() - 1) // 2
            bucket = st["buckets"][off.clamp(-R, R) + R].long()
        heads = 1 if G > chunk else max(1, min(Hkv, (1 << 28) // (Nq * Nk * G)))   # key heads at a time
        for h0 in range(0, Hkv, heads):
            kvs = slice(h0, min(h0 + heads, Hkv))
            for g0 in range(0, G, chunk):
                hs = [h * G + g for h in range(kvs.start, kvs.stop) for g in range(g0, min(g0 + chunk, G))]
                n_g = len(hs) // (kvs.stop - kvs.start)
                qq = q[b, hs].float()
                kk = k[b, kvs].float().repeat_interleave(n_g, 0)
                vv = v[b, kvs].float().repeat_interleave(n_g, 0)
                z = (qq @ kk.transpose(1, 2)) * st["scale"]
                if cap > 0:
                    t = torch.tanh(z / cap)
                    z = cap * t
                if st["slopes"] is not None:
                    z = z - st["slopes"][hs][:, None, None] * off.abs()
                if st["table"] is not None:
                    z = z + st["table"][hs].float()[:, bucket]
                see = vis
                if st["mask"] is not None:
                    kept = st["mask"][hs].repeat_interleave(BLOCK, 1)[:, :Nq].repeat_interleave(BLOCK, 2)[:, :, :Nk]
                    see = vis & (kept != 0)
                z = z.masked_fill(~see, NEG)
                mx = z.amax(-1, keepdim=True)
                mx = torch.where(mx == NEG, torch.zeros_like(mx), mx)
                p = torch.exp(z - mx)
                l = p.sum(-1, keepdim=True)
                p = p / torch.where(l == 0, torch.ones_like(l), l)
                oo = p @ vv
                o[b, hs] = oo.to(q.dtype)
                lse[b, hs] = (mx + torch.log(l)).squeeze(-1)
                if not train:
                    continue
                dd = do[b, hs].float()
                dp = dd @ vv.transpose(1, 2)
                ds = p * (dp - (dd * oo).sum(-1, keepdim=True))
                dv32[b, kvs] += (p.transpose(1, 2) @ dd).view(-1, n_g, Nk, d).sum(1)
                if st["table"] is not None:
                    # sums over the diagonals (row i shifted by i), then over the diagonals of a bucket
                    diag = torch.zeros(len(hs), Nq, Nk + Nq, device="cuda")
                    diag[:, :, :Nk] = ds.flip(1)
                    per = diag.view(len(hs), -1)[:, :Nq * (Nk + Nq - 1)].view(len(hs), Nq, Nk + Nq - 1)
                    per = per.sum(1, dtype=torch.float64)                    # column c: offset c - (Nq - 1)
                    offs = torch.arange(Nk + Nq - 1, device="cuda") - (Nq - 1) - st["q_start"][b]
                    dtable[hs] += torch.zeros(len(hs), st["table"].shape[1], device="cuda", dtype=torch.float64
                                              ).index_add_(1, st["buckets"][offs.clamp(-R, R) + R].long(), per)
                    del diag, per
                if cap > 0:
                    ds = ds * (1 - t * t)
                ds = ds * st["scale"]
                dq[b, hs] = (ds @ kk).to(q.dtype)
                dk32[b, kvs] += (ds.transpose(1, 2) @ qq).view(-1, n_g, Nk, d).sum(1)
    out = {"o": o, "lse": lse}
    if train:
        out.update(dq=dq, dk=dk32.to(k.dtype), dv=dv32.to(v.dtype))
        if st["table"] is not None:
            out["dtable"] = dtable.to(st["table"].dtype)
    return out


# ---- the definition in 64 bits --------------------------------------------------


def exact(case, seed):
    st = prepare(case, seed)
    lo, hi = (torch.from_numpy(x).cuda() for x in _intervals(case))
    B, H, Hkv, Nq, Nk, d = (case[k] for k in ("B", "H", "Hkv", "Nq", "Nk", "d"))
    train = case["kind"] == "train"
    blocks = None if st["mask"] is None else st["mask"].bool()
    keys = torch.arange(Nk, device="cuda")
    o = torch.zeros(B, H, Nq, d, device="cuda", dtype=torch.float64)
    lse = torch.full((B, H, Nq), NEG, device="cuda", dtype=torch.float64)
    out = {"o": o, "lse": lse}
    if train:
        out["dq"] = torch.zeros(B, H, Nq, d, device="cuda", dtype=torch.float64)
        out["dk"] = torch.zeros(B, Hkv, Nk, d, device="cuda", dtype=torch.float64)
        out["dv"] = torch.zeros(B, Hkv, Nk, d, device="cuda", dtype=torch.float64)
        if case["buckets"]:
            out["dtable"] = torch.zeros(H, case["buckets"], device="cuda", dtype=torch.float64)
    step = max(1, (1 << 26) // Nk)
    for b in range(B):
        pos0 = int(st["q_start"][b])
        for h in range(H):
            hk = h * Hkv // H
            K = st["k"][b, hk].double()
            V = st["v"][b, hk].double()
            for r0 in range(0, Nq, step):
                r1 = min(Nq, r0 + step)
                rows = torch.arange(r0, r1, device="cuda")
                see = (keys >= lo[b, r0:r1, None]) & (keys < hi[b, r0:r1, None])
                if blocks is not None:
                    see = see & blocks[h][rows // BLOCK][:, keys // BLOCK]
                Q = st["q"][b, h, r0:r1].double()
                rel = keys - (rows[:, None] + pos0)
                raw = torch.einsum("id,jd->ij", Q, K) * st["scale"]
                z = raw
                if case["cap"] > 0:
                    u = torch.exp(-2.0 * raw.abs() / case["cap"])
                    th = torch.sign(raw) * (1.0 - u) / (1.0 + u)
                    z = case["cap"] * th
                if st["slopes"] is not None:
                    z = z - st["slopes"][h].double() * rel.abs().double()
                if st["table"] is not None:
                    R = case["distance"]
                    bk = st["buckets"][torch.clamp(rel, -R, R) + R].long()
                    z = z + torch.take(st["table"][h].double(), bk)
                z = torch.where(see, z, torch.full_like(z, NEG))
                L = torch.logsumexp(z, 1)
                some = see.any(1)
                P = torch.where(see, torch.exp(z - torch.where(some, L, torch.zeros_like(L))[:, None]),
                                torch.zeros_like(z))
                O = torch.einsum("ij,jd->id", P, V)
                o[b, h, r0:r1] = O
                lse[b, h, r0:r1] = torch.where(some, L, torch.full_like(L, NEG))
                if not train:
                    continue
                dO = st["do"][b, h, r0:r1].double()
                out["dv"][b, hk] += torch.einsum("ij,id->jd", P, dO)
                dP = torch.einsum("id,jd->ij", dO, V)
                dZ = P * (dP - torch.einsum("ij,ij->i", P, dP)[:, None])
                if case["buckets"]:
                    for n in range(case["buckets"]):
                        out["dtable"][h, n] += torch.where(bk == n, dZ, torch.zeros_like(dZ)).sum()
                if case["cap"] > 0:
                    dZ = dZ * 4.0 * u / (1.0 + u) ** 2
                out["dq"][b, h, r0:r1] = torch.einsum("ij,jd->id", dZ, K) * st["scale"]
                out["dk"][b, hk] += torch.einsum("ij,id->jd", dZ, Q) * st["scale"]
    return out
