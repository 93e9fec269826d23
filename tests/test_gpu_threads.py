"""Calls from a host thread that has done no CUDA work yet (a loader's or a
server's worker, the autograd engine): no context is current there."""

import threading

import pytest
import torch

import block_sparse_attention_cross_b200 as cba
from tests._score_util import Case

pytestmark = pytest.mark.gpu


def _in_thread(call):
    got = []

    def run():
        try:
            got.append(call())
        except Exception as e:   # noqa: BLE001
            got.append(e)

    t = threading.Thread(target=run)
    t.start()
    t.join()
    if isinstance(got[0], Exception):
        raise got[0]
    return got[0]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_score_attention_from_a_new_thread(dtype):
    c = Case(H=2, Nq=150, d=64, dtype=dtype, cap=5.0, buckets=8, distance=30)
    want = c.run(True)
    kw, sp = c.score_kw(), c.spans()
    q, k, v, do = (c.gpu(x) for x in (c.q, c.k, c.v, c.do))
    torch.cuda.synchronize()
    o, lse = _in_thread(lambda: cba.score_attn_fwd(q, k, v, sp, return_lse=True, **kw))
    grads = _in_thread(lambda: cba.score_attn_bwd(do, q, k, v, o, lse, sp, **kw))
    torch.cuda.synchronize()
    for name, x in zip(("o", "lse", "dq", "dk", "dv", "dtable"), (o, lse, *grads)):
        assert torch.equal(x, want[name]), name


def test_block_sparse_attention_from_a_new_thread():
    g = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn(1, 2, 256, 64, generator=g).to(torch.bfloat16).cuda() for _ in range(3))
    bl = cba.compile(torch.ones(2, 2, 2, dtype=torch.uint8, device="cuda"))
    want = cba.sparse_attn_fwd(q, k, v, bl, 250)
    torch.cuda.synchronize()
    got = _in_thread(lambda: cba.sparse_attn_fwd(q, k, v, bl, 250))
    energy = _in_thread(lambda: cba.block_energy(q[0], k[0], 250))
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(energy, cba.block_energy(q[0], k[0], 250))
