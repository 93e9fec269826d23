"""The narrow checks of the score-modified attention are themselves checked, on
the CPU: an emulation of the kernels' roundings passes, and every result with a
term, a row group or a tile missing is refused."""

import numpy as np
import pytest
import torch

from tests._score_check import Narrow

BF, F32 = torch.bfloat16, torch.float32


def _round(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dtype).double().numpy()


def _emulate(c, ref, drop=()):
    """The results with the roundings that the kernels make; ``drop`` names what a wrong kernel leaves out."""
    B, H, Hkv, Nq, Nk, d = c.sizes
    q, k, v, do = (x.double().numpy() for x in (c.q, c.k, c.v, c.do))
    out = {n: np.zeros_like(ref[n]) for n in ("o", "dq", "dk", "dv", "dtable") if n in ref}
    out["lse"] = np.asarray(ref["lse"], np.float32)
    low = BF if c.dtype == BF else F32
    for b in range(B):
        pos = np.arange(Nq) + int((c.rules.get("q_start") or [0] * B)[b])
        off = np.arange(Nk)[None] - pos[:, None]
        for h in range(H):
            g = h // (H // Hkv)
            P = np.asarray(ref["P"][b, h], np.float32).astype(np.float64)
            if "tile" in drop:      # the last 64 keys of the first 64 rows
                P = P.copy()
                P[:64, -64:] = 0
            dP = np.asarray(ref["dP"][b, h], np.float32).astype(np.float64)
            D = 0.0 if "D" in drop else (P * dP).sum(1, keepdims=True)
            dZ = P * (dP - D)
            t = np.tanh(c.scale * (q[b, h] @ k[b, g].T) / c.cap) if c.cap > 0 and "factor" not in drop else 0.0
            dS = _round(dZ * (1 - t * t), low)
            out["o"][b, h] = _round(P, low) @ v[b, g]
            out["dq"][b, h] = c.scale * dS @ k[b, g]
            out["dk"][b, g] += c.scale * dS.T @ q[b, h]
            out["dv"][b, g] += _round(P, low).T @ do[b, h]
            if c.table is not None:
                R = len(c.buckets) // 2
                np.add.at(out["dtable"][h], c.buckets.numpy()[np.clip(off, -R, R) + R].ravel(), dZ.ravel())
    for n in out:
        if n != "lse":
            out[n] = _round(out[n], c.dtype)
    if "rows" in drop:              # a warp's rows of every head
        for n in ("o", "dq", "dk", "dv"):
            out[n][..., 32:64, :] = 0
    if "table" in drop and "dtable" in out:
        out["dtable"][:] = 0
    return out


CASES = [dict(Nq=300, d=64), dict(Nq=300, d=128, cap=5.0), dict(Nq=200, d=64, cap=2.0, slopes=True, buckets=6, distance=40, causal=True),
         dict(H=4, Hkv=2, Nq=260, d=64, buckets=32, distance=200), dict(Nq=150, d=64, cap=1e6), dict(Nq=260, d=64, scale=4.0, gain=6.0)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kw", CASES)
def test_roundings_pass(dtype, kw):
    c = Narrow(dtype=dtype, **kw)
    ref = c.reference(True)
    assert c.faults(_emulate(c, ref), ref) == []


def _drops():
    for kw in CASES:
        steep = "gain" in kw        # (one key a row: dS = 0 wherever D matters, and a lost tile may hold no probability)
        if not steep:
            yield kw, "D", "dq dk" + " dtable" * ("buckets" in kw)
        if 0 < kw.get("cap", 0) < 10:
            yield kw, "factor", "dq dk"
        yield kw, "rows", "o dq dk dv"
        if not steep and not kw.get("causal"):
            yield kw, "tile", "o dq dk dv"
        if "buckets" in kw:
            yield kw, "table", "dtable"


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kw,drop,names", list(_drops()))
def test_missing_parts_are_refused(dtype, kw, drop, names):
    c = Narrow(dtype=dtype, **kw)
    ref = c.reference(True)
    said = " ".join(c.faults(_emulate(c, ref, (drop,)), ref))
    for n in names.split():
        assert f"{n}:" in said, n


# (under a cap of 1e-5 s / cap is about 1e5, and its fp32 rounding alone moves the few scores whose factor 1 - tanh^2 is not 0
# by about 1: dQ and dK have no digits there, O and dV do.  Scores of 1e4 leave every row one key and dS = 0.)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cap,scale,gain,names", [(1e-5, 0.125, 1.0, "o dv"), (1e6, 0.125, 1.0, "o dq dk dv"), (1e4, 0.125, 1.0, "o dq dk dv"),
                                                  (1e5, 4000.0, 1e-4, "o dq dk dv")])
def test_zeros_are_refused_at_every_cap(dtype, cap, scale, gain, names):
    c = Narrow(H=1, Nq=150, d=64, dtype=dtype, cap=cap, scale=scale, gain=gain)
    ref = c.reference(True)
    zero = {n: np.zeros_like(ref[n]) for n in ("o", "dq", "dk", "dv")}
    said = " ".join(c.faults({**zero, "lse": ref["lse"]}, ref))
    for n in names.split():
        assert f"{n}:" in said, n
