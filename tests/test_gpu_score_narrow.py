"""Score-modified attention on the GPU against the float64 oracle, within the
narrow limits of tests/_score_check.py (which refuse a missing term, tile or
group of rows)."""

import numpy as np
import pytest
import torch

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
