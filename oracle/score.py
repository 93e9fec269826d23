"""Score-modified attention and its gradients in float64 (dense matrices, one
head at a time): capped scores, distance bias, learned bucket bias, intervals
of visible keys and kept blocks."""

from __future__ import annotations

import numpy as np


def spans(B, Nq, Nk, causal=False, docs=None, prefix=None, kv_len=None, q_len=None, q_start=None):
    """bool [B, Nq, Nk]: which keys every query row sees, pair by pair from the rules."""
    vis = np.zeros((B, Nq, Nk), dtype=bool)
    for b in range(B):
        kv = Nk if kv_len is None else int(kv_len[b])
        nq = Nq if q_len is None else int(q_len[b])
        p0 = 0 if q_start is None else int(q_start[b])
        doc_of = {}
        if docs is not None:
            for m in range(len(docs[b]) - 1):
                for x in range(int(docs[b][m]), int(docs[b][m + 1])):
                    doc_of[x] = m
        for i in range(min(nq, Nq)):
            p = p0 + i
            m = 0
            if docs is not None:
                if p not in doc_of:
                    continue
                m = doc_of[p]
            for j in range(min(kv, Nk)):
                if docs is not None and doc_of.get(j) != m:
                    continue
                if causal and j > p:
                    start = 0 if docs is None else int(docs[b][m])
                    if prefix is None or j >= start + int(prefix[b][m]):
                        continue
                vis[b, i, j] = True
    return vis


def relative_bucket(off, n_buckets, max_distance, bidirectional):
    """Bucket of offset ``off`` = key - query, in integer arithmetic: the largest t with
    (x / e)^m >= (max_distance / e)^t, where m logarithmic buckets follow the e exact ones."""
    half = n_buckets // 2 if bidirectional else n_buckets
    base = half if bidirectional and off > 0 else 0
    if not bidirectional and off > 0:
        return 0
    x = abs(off)
    e = half // 2
    if x < e:
        return base + x
    m = half - e
    t = 0
    while t < m and x ** m * e ** (t + 1) >= max_distance ** (t + 1) * e ** m:
        t += 1
    return base + min(half - 1, e + t)


def score_attention(q, k, v, vis, scale, cap=0.0, slopes=None, table=None, buckets=None, mask=None, block=128,
                    q_start=None, dout=None):
    """O, LSE and, with ``dout``, the gradients.  q [B, H, Nq, d]; k, v [B, Hkv, Nk, d]; float64.

    Also returns, per head, what error bounds need: P, dP, the factor of the
    cap and dS as lists over (b, h)."""
    B, H, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    out = {"o": np.zeros((B, H, Nq, d)), "lse": np.full((B, H, Nq), -np.inf), "P": {}}
    if dout is not None:
        out.update(dq=np.zeros_like(q), dk=np.zeros_like(k), dv=np.zeros_like(v), dP={}, dZ={}, dS={})
        if table is not None:
            out["dtable"] = np.zeros(table.shape)
    for b in range(B):
        pos = np.arange(Nq) + (0 if q_start is None else int(q_start[b]))
        off = np.arange(Nk)[None, :] - pos[:, None]
        for h in range(H):
            g = h // (H // Hkv)
            z = scale * (q[b, h] @ k[b, g].T)
            th = np.zeros_like(z)
            if cap > 0:
                th = np.tanh(z / cap)
                z = cap * th
            if slopes is not None:
                z = z - slopes[h] * np.abs(off)
            if table is not None:
                R = len(buckets) // 2
                bk = np.asarray(buckets)[np.clip(off, -R, R) + R]
                z = z + table[h][bk]
            see = vis[b].copy()
            if mask is not None:
                see &= np.kron(mask[h], np.ones((block, block)))[:Nq, :Nk] != 0
            some = see.any(1)
            z = np.where(see, z, -np.inf)
            mx = np.where(some, z.max(1), 0.0)
            e = np.where(see, np.exp(z - mx[:, None]), 0.0)
            l = e.sum(1)
            P = e / np.where(some, l, 1.0)[:, None]
            with np.errstate(divide="ignore"):
                out["lse"][b, h] = np.where(some, mx + np.log(l), -np.inf)
            out["o"][b, h] = P @ v[b, g]
            out["P"][b, h] = P
            if dout is None:
                continue
            dP = dout[b, h] @ v[b, g].T
            dZ = P * (dP - (P * dP).sum(1, keepdims=True))
            dS = dZ * (1 - th * th) * scale
            out["dv"][b, g] += P.T @ dout[b, h]
            out["dq"][b, h] = dS @ k[b, g]
            out["dk"][b, g] += dS.T @ q[b, h]
            if table is not None:
                np.add.at(out["dtable"][h], bk.ravel(), dZ.ravel())
            out["dP"][b, h], out["dZ"][b, h], out["dS"][b, h] = dP, dZ, dS
    return out
