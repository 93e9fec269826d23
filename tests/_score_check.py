"""Narrow checks of the score-modified attention, beside the elementwise bounds
of tests/_score_util.py.

``Narrow.verify`` compares with the float64 oracle twice.

* Elementwise, worst case.  The errors are those of tests/_score_util.py, taken
  where they arise (u: half a step, bf16 2^-8, fp32 2^-24):
  a capped score is off by 16 2^-24 of itself (the cap adds no error of its own
  size to a small score); P_ij by its own error and the P-weighted mean of its
  row's; and in bf16 D is the kernel's sum of P dP in fp32, not dO . O.
* By norms, of every tensor and of every group of 32 rows of a head.  The
  roundings to bf16 of P and dS are independent: an element of a product with
  them is off by the root of the sum of squares, each at most u and u / sqrt(3)
  in the mean square.  A group's error may be twice that: one rounding alone
  reaches at most sqrt(3) of it, many concentrate at it.  The fp32 errors enter
  as random ones too (a dot product: 8 2^-24 of its absolute sum), four times.
  A wrong row, tile or term leaves these limits although it may stay within the
  worst case of every element.
"""

import numpy as np
import torch

from tests._score_util import F24, Case

GROUP = 32


class Narrow(Case):
    def _limits(self, ref, train):
        """Per tensor: worst error of every element, and the variances of its bf16 and fp32 errors."""
        B, H, Hkv, Nq, Nk, d = self.sizes
        bf = self.dtype == torch.bfloat16
        u = 2.0 ** -8 if bf else F24
        q, k, v, do = (x.double().numpy() for x in (self.q, self.k, self.v, self.do))
        shapes = {"o": q.shape, "lse": q.shape[:3]}
        if train:
            shapes.update(dq=q.shape, dk=k.shape, dv=v.shape)
            if self.table is not None:
                shapes["dtable"] = tuple(self.table.shape)
        worst, vb, vf = ({n: np.zeros(s) for n, s in shapes.items()} for _ in range(3))
        c2 = u * u / 3
        table = None if self.table is None else self.table.double().numpy()
        for b in range(B):
            pos = np.arange(Nq) + int((self.rules.get("q_start") or [0] * B)[b])
            off = np.arange(Nk)[None] - pos[:, None]
            for h in range(H):
                g = h // (H // Hkv)
                P = ref["P"][b, h]
                s = self.scale * (q[b, h] @ k[b, g].T)
                zabs = self.scale * (np.abs(q[b, h]) @ np.abs(k[b, g]).T)
                t = np.tanh(s / self.cap) if self.cap > 0 else np.zeros_like(s)
                c = self.cap * t if self.cap > 0 else s
                bias, size = np.zeros_like(s), np.zeros_like(s)
                if self.slopes is not None:
                    bias = bias - float(self.slopes[h]) * np.abs(off)
                    size = size + np.abs(bias)
                if table is not None:
                    R = len(self.buckets) // 2
                    bk = self.buckets.numpy()[np.clip(off, -R, R) + R]
                    bias = bias + table[h][bk]
                    size = size + np.abs(table[h][bk])
                z = c + bias
                lse = np.where(np.isfinite(ref["lse"][b, h]), ref["lse"][b, h], 0.0)[:, None]
                rest = 16 * (np.abs(c) + size) + 8 * (1 + np.abs(z) + np.abs(lse))
                on = P > 0
                ez = np.where(on, (d + 16) * zabs + rest, 0.0) * F24
                et = np.where(on, 8 * zabs + rest, 0.0) * F24
                e = ez + (P * ez).sum(1, keepdims=True) + Nk * F24
                row = np.sqrt((P * P * et * et).sum(1, keepdims=True)) + 8 * F24     # common to a row
                o = ref["o"][b, h]
                worst["o"][b, h] = ((u + e) * P) @ np.abs(v[b, g]) + 2 * u * np.abs(o)
                vb["o"][b, h] = (c2 * P * P if bf else 0 * P) @ v[b, g] ** 2 + 2 * c2 * o * o
                vf["o"][b, h] = (P * P * (et + 8 * F24) ** 2) @ v[b, g] ** 2 + (row * o) ** 2
                worst["lse"][b, h] = (P * ez).sum(1) + (Nk + 4 * np.abs(lse[:, 0]) + 4) * F24
                vf["lse"][b, h] = (row[:, 0] + 4 * F24 * np.abs(lse[:, 0])) ** 2
                if not train:
                    continue
                dP, dZ, dS = ref["dP"][b, h], ref["dZ"][b, h], ref["dS"][b, h]
                adp = np.abs(do[b, h]) @ np.abs(v[b, g]).T
                D = (P * dP).sum(1, keepdims=True)
                f = (1 - t * t) * self.scale
                ef = self.scale * (2.0 ** -20 + 2 * (d + 16) * F24 * zabs / self.cap) if self.cap > 0 else 0.0
                if bf:
                    eD = (P * (e * np.abs(dP) + ((d + 4) * adp + Nk * np.abs(dP)) * F24)).sum(1, keepdims=True)
                else:
                    eD = (np.abs(do[b, h]) * (worst["o"][b, h] + d * F24 * np.abs(o))).sum(1, keepdims=True)
                tD = np.sqrt((P * P * ((et * dP) ** 2 + (8 * F24 * adp) ** 2)).sum(1, keepdims=True)) + 8 * F24 * (
                    P * np.abs(dP)).sum(1, keepdims=True)
                edZ = P * (eD + (d + 4) * F24 * adp + (e + 4 * F24) * np.abs(dP - D))
                tdZ = P * np.sqrt((8 * F24 * adp) ** 2 + ((et + 8 * F24) * (dP - D)) ** 2)   # and P tD, r dZ a row
                r = row + 4 * F24 * np.abs(lse)
                edS = edZ * (f + ef) + ef * np.abs(dZ) + (u + 8 * F24) * np.abs(dS)
                vS = (tdZ * f) ** 2 + (0.25 * ef * dZ) ** 2
                rS = P * f * tD + np.abs(dS) * r
                worst["dq"][b, h] = (edS + Nk * F24 * np.abs(dS)) @ np.abs(k[b, g]) + u * np.abs(ref["dq"][b, h])
                vb["dq"][b, h] = (c2 * dS * dS if bf else 0 * P) @ k[b, g] ** 2 + c2 * ref["dq"][b, h] ** 2
                vf["dq"][b, h] = vS @ k[b, g] ** 2 + (tD * ((P * f) @ k[b, g])) ** 2 + (r * ref["dq"][b, h]) ** 2
                worst["dk"][b, g] += (edS + Nq * F24 * np.abs(dS)).T @ np.abs(q[b, h])
                vb["dk"][b, g] += (c2 * dS * dS if bf else 0 * P).T @ q[b, h] ** 2
                vf["dk"][b, g] += (vS + rS * rS).T @ q[b, h] ** 2
                worst["dv"][b, g] += ((u + e + Nq * F24) * P).T @ np.abs(do[b, h])
                vb["dv"][b, g] += (c2 * P * P if bf else 0 * P).T @ do[b, h] ** 2
                vf["dv"][b, g] += (P * P * ((et + 8 * F24) ** 2 + r * r)).T @ do[b, h] ** 2
                if table is not None:
                    np.add.at(worst["dtable"][h], bk.ravel(), (edZ + 64 * F24 * np.abs(dZ)).ravel())
                    np.add.at(vf["dtable"][h], bk.ravel(), (tdZ ** 2 + (8 * F24 * dZ) ** 2).ravel())
                    # what a row's D and LSE put into all its pairs of a bucket
                    for n in range(table.shape[1]):
                        at = bk == n
                        vf["dtable"][h, n] += ((tD[:, 0] * (P * at).sum(1)) ** 2 + (r[:, 0] * (dZ * at).sum(1)) ** 2).sum()
        if train:
            for n in ("dk", "dv", "dtable"):
                if n in worst:
                    worst[n] += u * np.abs(ref[n])
                    vb[n] += c2 * ref[n] ** 2
        return worst, vb, vf

    def faults(self, got, ref, train=True):
        """What of ``got`` is beyond the limits, as texts."""
        worst, vb, vf = self._limits(ref, train)
        bad = []
        for n, w in worst.items():
            x, y = np.asarray(got[n], dtype=np.float64), ref[n]
            if n == "lse":
                dead = np.isneginf(y)
                if not np.array_equal(np.isneginf(x), dead):
                    bad.append("lse: rows that see nothing differ")
                x, y = np.where(dead, 0, x), np.where(dead, 0, y)
            err = np.abs(x - y)
            if not np.isfinite(x).all():
                bad.append(f"{n}: not finite")
                continue
            over = err > 1.01 * w + 1e-30
            if over.any():
                bad.append(f"{n}: {over.sum()} of {over.size} elements beyond the bound, worst "
                           f"{(err / np.maximum(w, 1e-300)).max():.3g} times")
            if n == "lse":
                continue
            rows = {"dtable": 1}.get(n, GROUP)
            flat = [a.reshape(-1, *a.shape[-2:]) if n != "dtable" else a[:, None, :] for a in (err, vb[n], vf[n])]
            for head in range(flat[0].shape[0]):
                for r0 in range(0, flat[0].shape[1], rows):
                    e2, b2, f2 = (float((a[head, r0:r0 + rows] ** p).sum()) for a, p in zip(flat, (2, 1, 1)))
                    if e2 ** 0.5 > 2 * b2 ** 0.5 + 4 * f2 ** 0.5 + 1e-30:
                        bad.append(f"{n}: head {head} rows {r0}..: norm of the error {e2 ** 0.5:.3e} beyond 2 x {b2 ** 0.5:.3e}"
                                   f" + 4 x {f2 ** 0.5:.3e}")
        return bad

    def verify(self, train=True):
        got = {n: x.double().cpu().numpy() for n, x in self.run(train).items()}
        ref = self.reference(train)
        bad = self.faults(got, ref, train)
        assert not bad, bad[:8]
        return got, ref
