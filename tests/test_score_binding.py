"""Integers of the score-modified attention's binding beyond the C interface's
int are refused or clamped, never wrapped into range.  CPU only."""

import numpy as np
import pytest
import torch

import block_sparse_attention_cross_b200 as cba
from block_sparse_attention_cross_b200 import score


@pytest.mark.parametrize("n,dist", [(4, (1 << 32) + 2), ((1 << 32) + 4, 2), (4, (1 << 40) + 2), (4, -(1 << 32) + 2), (-(1 << 32) + 4, 2)])
def test_bucket_sizes_do_not_wrap(n, dist):
    with pytest.raises(cba.CalibattError):
        cba.relative_buckets(n, dist, True, device="cpu")


@pytest.mark.parametrize("sizes", [((1 << 32) + 1, 4, 4), (1, (1 << 32) + 4, 4), (1, 4, (1 << 32) + 4)])
def test_span_sizes_do_not_wrap(sizes):
    with pytest.raises(ValueError, match="2\\^31"):
        cba.attn_spans(*sizes, device="cuda:0")


@pytest.mark.parametrize("values,want", [
    (np.array([3_000_000_000, 7], np.uint32), [(1 << 31) - 1, 7]),
    (np.array([(1 << 63) + 5, 7], np.uint64), [(1 << 31) - 1, 7]),
    (np.array([1 << 40, -(1 << 40)], np.int64), [(1 << 31) - 1, -(1 << 31)]),
    (np.array([200, 7], np.uint8), [200, 7]),
])
def test_lengths_do_not_wrap(values, want):
    got = score._ints("x", values, (2,), torch.device("cpu"))
    assert got.dtype == torch.int32 and got.tolist() == want


def test_map_offset_does_not_wrap():
    assert score._int32((1 << 32) + 3) == (1 << 31) - 1 and score._int32(-(1 << 32)) == -(1 << 31) and score._int32(5) == 5
