"""Writes into a cache held in 8 bits: scales at the end of the range, and captured calls, on the GPU."""
import pytest
import torch

import q8_helpers as Q
from gpu_helpers import pkv
from test_gpu_q8 import Write

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def P():
    m = pkv()
    m.pkv_get_device_error()
    return m


@pytest.mark.parametrize("T", [3, 1100])
@pytest.mark.parametrize("power", [126, 127])
def test_write_into_pages_of_the_largest_scales(P, T, power):
    # scales of 2^126 and 2^127, whose reciprocals are the least normal number and half of it
    w = Write([(3, T)], 2, 2, 64, 16, torch.bfloat16, seed=power, norm=False, rot=0)
    _, k, v = w.rows(w.x)
    for x in (k, v):
        x.copy_((x.float().clamp(-1.9, 1.9) * 2.0 ** 127).to(torch.bfloat16))
    w.ks[:], w.vs[:] = 2.0 ** power, 2.0 ** power
    w.run(P)
    blk, row = w.slots // 16, w.slots % 16
    first = blk == blk[0]       # the block that was begun before: its scale is the larger one
    for x, codes, scale in ((k, w.gpu[0], w.gpu[2]), (v, w.gpu[1], w.gpu[3])):
        assert bool((scale[blk[0]] == 2.0 ** power).all())
        got = codes.cpu().double()[blk[first], :, row[first]]
        assert torch.equal(got, Q.code_of(x[first].double() / 2.0 ** power))
        if T > 16:
            s = scale.cpu().double()[blk[~first]][:, :, None]
            assert torch.equal(codes.cpu().double()[blk[~first], :, row[~first]], Q.code_of(x[~first].double() / s))
    assert P.pkv_get_device_error() == 0


@pytest.mark.parametrize("T", [40, 1500])
def test_write_captured_and_called(P, T):
    # a captured write, replayed, leaves the bits that the call leaves
    w = Write([(0, T - 30), (7, 29), (30, 1)], 8, 2, 128, 16, torch.bfloat16, seed=T)
    w.run(P)
    w.check()
    x, table = w.x.to(DEV), w.cos_sin.to(DEV)
    q, k, v = w.rows(x)
    caches = [t.to(DEV) for t in (w.kc, w.vc, w.ks, w.vs)]
    begin = [t.clone() for t in caches]
    q_out, pos, slots = torch.zeros_like(w.q_out), w.pos.to(DEV), w.slots.to(DEV)
    wq, wk = w.wq.to(DEV), w.wk.to(DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        P.pkv_qk_norm_rope_write_q8(q, k, v, *caches, pos, slots, q_out, q_weight=wq, k_weight=wk, eps=w.eps,
                                    cos_sin=table)
    for _ in range(3):
        for a, b in zip(caches, begin):
            a.view(torch.uint8).copy_(b.view(torch.uint8))
        q_out.zero_()
        graph.replay()
        assert torch.equal(q_out, w.q_out)
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(caches, w.gpu))
    assert P.pkv_get_device_error() == 0
