"""Attention over a cache held in 8 bits with workspaces and limits made for larger calls, on the GPU."""
import pytest
import torch

from gpu_helpers import pkv
from test_gpu_q8 import Decode
from test_gpu_q8_chunk import MIXED, Chunk

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def P():
    m = pkv()
    m.pkv_get_device_error()
    return m


@pytest.mark.parametrize("Hq,Hkv,NQ,longest", [(32, 8, 1, 8192), (16, 2, 3, 9000), (40, 40, 1, 5000)])
def test_decode_in_the_workspace_of_the_largest_batch(P, Hq, Hkv, NQ, longest):
    # requests leave one after another, and the longest first: the same workspace, poisoned each time
    lens = [longest] + [40 + (i * 911) % 3000 for i in range(39)]
    d = Decode(lens, NQ, Hq, Hkv, 64, 16, torch.bfloat16, seed=Hq)
    kc, vc, ks, vs = (t.to(DEV) for t in (d.kc, d.vc, d.ks, d.vs))
    ws = P.workspace_tensor(P.pkv_decode_q8_workspace_bytes(kc, 40, NQ, Hq, longest), DEV)
    want = d.run(P)
    d.check(want)
    ref, mean, _, _, _ = d.want()
    q, tables, ctx = d.q.to(DEV), d.tables.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    for first, last, limit in ((0, 40, longest), (0, 20, longest), (0, 9, longest), (0, 8, longest), (0, 4, longest),
                               (0, 1, longest), (1, 40, longest), (1, 5, 4500), (1, 2, longest), (30, 40, 3100)):
        out = torch.full(d.q[first:last].shape, 9.0, dtype=d.dt, device=DEV)
        ws.fill_(0xff)
        P.pkv_paged_attention_decode_q8(q[first:last].contiguous(), kc, vc, ks, vs, tables[first:last].contiguous(),
                                        ctx[first:last].contiguous(), d.scale, out, limit, 0, ws)
        # cut in other places: each within the output's rounding and 2^-11 of the weights of the other
        rows = slice(first * NQ, last * NQ)
        tol = (2.0 ** -10 * mean[rows] + 2 * 2.0 ** -8 * ref[rows].abs()) * 1.01 + 2.0 ** -20
        off = (out.cpu().view(-1, Hq, 64).double() - want[first:last].view(-1, Hq, 64).double()).abs()
        assert bool((off <= tol).all()), (first, last, limit)
    assert P.pkv_get_device_error() == 0


@pytest.mark.parametrize("limit", [700, 4097, 40000, 1 << 20])
def test_decode_with_a_limit_far_above_the_contexts(P, limit):
    # what a captured step passes: the model's longest context, not the batch's
    d = Decode([700, 1, 0, 333, 64, 129], 2, 8, 2, 128, 16, torch.float16, seed=4)
    for out_dtype in (torch.float16, torch.float32):
        d.check(d.run(P, out_dtype, max_ctx=limit))
    assert P.pkv_get_device_error() == 0


@pytest.mark.parametrize("limit", [764, 40000, 1 << 20])
def test_chunk_with_a_limit_far_above_the_contexts(P, limit):
    for dt in (torch.float16, torch.bfloat16):
        c = Chunk(MIXED, 8, 2, 128, 16, dt, seed=2, room=3)
        c.check(c.run(P, max_ctx=limit))
        c.check(c.run(P, torch.float32, max_ctx=limit))
    assert P.pkv_get_device_error() == 0
