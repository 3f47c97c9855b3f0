"""Decode over a cache held in 8 bits: rows without a good block, and rows without a finite score, on the GPU."""
import pytest
import torch

import q8_helpers as Q
from gpu_helpers import pkv
from test_gpu_q8 import Decode
from test_gpu_q8_edges import MANY

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    m = pkv()
    m.pkv_get_device_error()
    return m


@pytest.mark.parametrize("part", [0, 16, 64])
@pytest.mark.parametrize("lens,Hq,Hkv,NQ", [([40, 300, 16], 4, 2, 1), ([40, 300, 16], 8, 2, 3), (MANY, 16, 2, 3)])
def test_decode_of_contexts_without_a_good_block(P, lens, Hq, Hkv, NQ, part):
    # a row all of whose positions are left out sees nothing, and is zero
    d = Decode(lens, NQ, Hq, Hkv, 64, 16, torch.float16, seed=1)
    good = d.run(P, torch.float32, part)
    d.tables[1] = -1
    out = d.run(P, torch.float32, part)
    assert P.pkv_get_device_error() == P.DEVERR["BLOCK_ID"]
    assert bool((out[1] == 0).all())
    assert torch.equal(out[0], good[0]) and torch.equal(out[2:], good[2:])


def test_decode_of_queries_whose_only_good_block_is_later(P):
    # 17 positions, three queries: the second block is good, and only the last query sees into it
    d = Decode([17], 3, 4, 2, 64, 16, torch.float16, seed=2)
    d.tables[0, 0] = -1
    out = d.run(P, torch.float32)
    assert P.pkv_get_device_error() == P.DEVERR["BLOCK_ID"]
    blk = int(d.tables[0, 1])
    v = Q.numbers(d.vc, d.vs)[blk, :, 0].repeat_interleave(2, 0)
    assert bool((out[0, :2] == 0).all())
    assert bool(((out[0, 2].double() - v).abs() <= 2.0 ** -22 * v.abs()).all())


@pytest.mark.parametrize("part", [0, 16])
def test_decode_of_scores_below_the_range(P, part):
    # all scores -inf, with every block good: no weight, and not the zero of a row that sees nothing
    d = Decode([70, 40], 1, 4, 2, 64, 16, torch.bfloat16, seed=3)
    d.q[0] = -2.0 ** 100
    d.kc[:] = torch.tensor(448.0).to(Q.CODE)
    d.ks[:] = 2.0 ** 60
    d.q[1] = 0
    out = d.run(P, part=part)
    assert bool(out[0].isnan().all()) and bool(torch.isfinite(out[1]).all())
    assert P.pkv_get_device_error() == 0
