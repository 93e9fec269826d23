"""Cases, inputs and derived error bounds of the score-modified attention tests.

Bounds, from the roundings that the kernels make (u = half a bf16 step
relative to the value = 2^-8, for fp32 2^-24; all elementwise, first order):

* scores: an fp32 dot product of d terms is off by at most (d + 16) 2^-24
  scale sum |q||k|, the bias terms and the cap (|z| up to cap, a few roundings
  of it) by 16 2^-24 of their size; exp and its argument add 8 2^-24 (1 + |z -
  max|).  ``ez`` is the sum: the relative error of a probability is at most
  2 ez (numerator and normaliser).
* O: probabilities rounded to u, the normaliser corrected for the largest one
  (at most u more), the result rounded to u.
* The cap's factor 1 - t^2 with |t| <= 1 rounded to fp32: t is off by at most
  2^-22 (MUFU exponential and reciprocal, 2 units in the last place each; a
  rounding of tanhf in fp32), so the factor is off by at most 2 |t| 2^-22 plus
  a rounding of 1, together below 2^-20, absolutely: where the cap saturates
  the factor itself is far smaller.  dS gets |dZ| scale 2^-20 from it.
* D = sum dO O inherits O's error; dZ = P (dP - D); dS rounded to u for its
  product; results rounded to u.  Sums of n terms in fp32 add n 2^-24 of the
  absolute sum, far below u in bf16 and part of ``ez`` in fp32.
"""

import math

import numpy as np
import torch

import block_sparse_attention_cross_b200 as cba
from oracle import score as osc

F24 = 2.0 ** -24


class Case:
    """Inputs on the host (float64, exactly the device's values) and on the GPU."""

    def __init__(self, B=1, H=2, Hkv=None, Nq=64, Nk=None, d=64, dtype=torch.bfloat16, cap=0.0, slopes=False, buckets=0,
                 distance=16, layout="bhnd", mask=None, seed=0, scale=None, gain=1.0, bidirectional=True, **rules):
        Hkv = H if Hkv is None else Hkv
        Nk = Nq if Nk is None else Nk
        self.sizes = (B, H, Hkv, Nq, Nk, d)
        self.dtype, self.cap, self.rules, self.d = dtype, cap, rules, d
        g = torch.Generator().manual_seed(1234 + seed)

        def acts(h, n, k=1.0):
            x = (torch.randn(B, n, h, d, generator=g) * k).to(dtype)
            return x.transpose(1, 2) if layout == "bnhd" else x.transpose(1, 2).contiguous()

        self.q, self.k, self.v, self.do = acts(H, Nq, gain), acts(Hkv, Nk), acts(Hkv, Nk), acts(H, Nq)
        self.scale = 1.0 / math.sqrt(d) if scale is None else scale
        self.slopes = torch.tensor([2.0 ** -(1 + h % 6) for h in range(H)]) if slopes else None
        self.table = torch.randn(H, buckets, generator=g).to(dtype) if buckets else None
        self.buckets = cba.relative_buckets(buckets, distance, bidirectional, device="cpu") if buckets else None
        self.mask = mask

    def gpu(self, x):
        # moves a tensor and keeps its strides
        if x is None:
            return None
        if x.dim() == 4 and not x.is_contiguous():
            return x.transpose(1, 2).cuda().transpose(1, 2)
        return x.cuda()

    def spans(self):
        B, _, _, Nq, Nk, _ = self.sizes
        return cba.attn_spans(B, Nq, Nk, **self.rules)

    def score_kw(self):
        return dict(scale=self.scale, cap=self.cap, slopes=self.gpu(self.slopes), table=self.gpu(self.table),
                    buckets=self.gpu(self.buckets), mask=self.gpu(self.mask))

    def reference(self, train):
        B, H, Hkv, Nq, Nk, d = self.sizes
        vis = osc.spans(B, Nq, Nk, **self.rules)
        n64 = lambda x: None if x is None else x.double().numpy()   # noqa: E731
        ref = osc.score_attention(n64(self.q), n64(self.k), n64(self.v), vis, float(np.float32(self.scale)), cap=self.cap,
                                  slopes=n64(self.slopes), table=n64(self.table),
                                  buckets=None if self.buckets is None else self.buckets.numpy(),
                                  mask=None if self.mask is None else self.mask.numpy(),
                                  q_start=self.rules.get("q_start"), dout=n64(self.do) if train else None)
        ref["vis"] = vis
        return ref

    def bounds(self, ref, train):
        B, H, Hkv, Nq, Nk, d = self.sizes
        u = 2.0 ** -8 if self.dtype == torch.bfloat16 else F24
        q, k, v, do = (x.double().numpy() for x in (self.q, self.k, self.v, self.do))
        out = {"o": np.zeros((B, H, Nq, d)), "lse": np.zeros((B, H, Nq))}
        if train:
            out.update(dq=np.zeros(q.shape), dk=np.zeros(k.shape), dv=np.zeros(v.shape))
            if self.table is not None:
                out["dtable"] = np.zeros(self.table.shape)
        big = max(float(np.abs(self.table.double().numpy()).max()) if self.table is not None else 0.0, 0.0)
        for b in range(B):
            pos = np.arange(Nq) + int((self.rules.get("q_start") or [0] * B)[b])
            off = np.arange(Nk)[None] - pos[:, None]
            for h in range(H):
                g = h // (H // Hkv)
                P = ref["P"][b, h]
                zabs = self.scale * (np.abs(q[b, h]) @ np.abs(k[b, g]).T)
                size = big + self.cap + (float(self.slopes[h]) * np.abs(off) if self.slopes is not None else 0.0)
                ez = ((d + 16) * zabs + 16 * size + 8 * (1 + zabs + size)) * F24
                ez = np.where(P > 0, ez, 0.0).max(1, keepdims=True) + Nk * F24
                e2 = 2 * ez
                absv = P @ np.abs(v[b, g])
                out["o"][b, h] = (2 * u + e2) * absv + 2 * u * np.abs(ref["o"][b, h])
                lse = ref["lse"][b, h]
                out["lse"][b, h] = np.where(np.isfinite(lse), e2[:, 0] + 4 * F24 * np.abs(lse), 0.0)
                if not train:
                    continue
                f = np.where(np.abs(ref["dZ"][b, h]) > 0, ref["dS"][b, h] / np.where(ref["dZ"][b, h] == 0, 1, ref["dZ"][b, h]),
                             self.scale)
                adp = np.abs(do[b, h]) @ np.abs(v[b, g]).T
                D = np.abs((P * ref["dP"][b, h]).sum(1, keepdims=True))
                eD = (np.abs(do[b, h]) * out["o"][b, h]).sum(1, keepdims=True) + d * F24 * (
                    np.abs(do[b, h]) * np.abs(ref["o"][b, h])).sum(1, keepdims=True)
                edZ = P * (eD + (d + 4) * F24 * adp + (e2 + 4 * F24) * (adp + D))
                ef = 2.0 ** -20 * self.scale if self.cap > 0 else 0.0
                edS = edZ * (f + ef) + (u + 8 * F24 + e2) * np.abs(ref["dS"][b, h]) + ef * np.abs(ref["dZ"][b, h])
                out["dq"][b, h] = edS @ np.abs(k[b, g]) + (u + Nk * F24) * np.abs(ref["dq"][b, h])
                out["dk"][b, g] += edS.T @ np.abs(q[b, h])
                out["dv"][b, g] += (((u + e2) * P).T + Nq * F24 * P.T) @ np.abs(do[b, h])
                if self.table is not None:
                    R = len(self.buckets) // 2
                    bk = self.buckets.numpy()[np.clip(off, -R, R) + R]
                    np.add.at(out["dtable"][h], bk.ravel(), (edZ + 64 * F24 * np.abs(ref["dZ"][b, h])).ravel())
        if train:
            out["dk"] += (u + Nq * F24) * np.abs(ref["dk"])
            out["dv"] += (u + Nq * F24) * np.abs(ref["dv"])
            if self.table is not None:
                out["dtable"] += u * np.abs(ref["dtable"])
        for name in out:
            if name != "lse":
                out[name] = out[name] * 1.01 + 1e-30   # second-order terms
        return out

    def run(self, train):
        kw = self.score_kw()
        q, k, v, do = (self.gpu(x) for x in (self.q, self.k, self.v, self.do))
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        sp = self.spans()
        o, lse = cba.score_attn_fwd(q, k, v, sp, return_lse=True, status=status, **kw)
        got = {"o": o, "lse": lse}
        if train:
            g = cba.score_attn_bwd(do, q, k, v, o, lse, sp, status=status, **kw)
            got.update(zip(("dq", "dk", "dv", "dtable"), g))
            assert g[0].stride() == q.stride() and g[1].stride() == k.stride()
        assert status.item() == 0
        return got

    def check(self, train=True):
        got = self.run(train)
        ref = self.reference(train)
        bound = self.bounds(ref, train)
        for name, b in bound.items():
            x, y = got[name].double().cpu().numpy(), ref[name]
            if name == "lse":
                dead = np.isneginf(y)
                assert np.array_equal(np.isneginf(x), dead), "rows that see nothing differ"
                x, y = np.where(dead, 0, x), np.where(dead, 0, y)
            err = np.abs(x - y)
            assert np.isfinite(x).all(), name
            bad = err > b
            assert not bad.any(), (f"{name}: {bad.sum()} of {bad.size} beyond the bound, worst "
                                   f"{(err / np.maximum(b, 1e-300)).max():.3g} times, max abs {err.max():.3e}")
        return got, ref
