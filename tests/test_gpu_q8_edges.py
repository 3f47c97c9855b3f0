"""Decode over a cache held in 8 bits: values that are NaN and not seen by every query, on the GPU."""
import pytest
import torch

import q8_helpers as Q
from gpu_helpers import pkv
from test_gpu_q8 import Decode

pytestmark = pytest.mark.gpu

DEV = "cuda"
NAN = torch.tensor([0x7f, 0xff], dtype=torch.uint8).view(Q.CODE)  # e4m3's two


@pytest.fixture(scope="module")
def P():
    m = pkv()
    m.pkv_get_device_error()
    return m


def _place(d, s, t):
    return int(d.tables[s, t // d.B]), t % d.B


FEW = [50, 49, 51, 300, 3, 2, 1, 67]                       # the last positions in one step and in two
MANY = [20 + (i * 53) % 90 for i in range(200)] + [2900]   # so many that a CTA takes 16 columns


@pytest.mark.parametrize("part", [0, 16, 64])
@pytest.mark.parametrize("lens,Hq,Hkv,NQ,D,B", [
    (FEW, 4, 2, 3, 64, 16), (FEW, 8, 2, 4, 128, 32), (FEW, 8, 1, 2, 128, 16), (MANY, 16, 2, 3, 64, 16),
    (MANY, 10, 1, 2, 128, 32)])
def test_decode_values_that_only_later_queries_see(P, lens, Hq, Hkv, NQ, D, B, part):
    # a NaN in the value of each of the last positions, an element and a code of its own: the queries that
    # see it have it in that element, and nothing else changes
    part = part * B // 16
    for out_dtype in (torch.float16, torch.float32):
        d = Decode(lens, NQ, Hq, Hkv, D, B, torch.float16, seed=NQ)
        want = d.run(P, out_dtype, part)
        G = Hq // Hkv
        for s, n in enumerate(lens):
            for j in range(NQ):
                t = n - NQ + j
                if t < 0:
                    continue
                h, e = (s + j) % Hkv, (7 * s + 13 * j) % D
                blk, row = _place(d, s, t)
                d.vc[blk, h, row, e] = NAN[(s + j) % 2]
                want[s, j:, h * G:(h + 1) * G, e] = float("nan")
        out = d.run(P, out_dtype, part)
        assert torch.equal(out.isnan(), want.isnan())
        assert torch.equal(torch.nan_to_num(out), torch.nan_to_num(want))
    assert P.pkv_get_device_error() == 0


def test_decode_steps_full_of_nan_values(P):
    # every element of the last positions, in both kv heads
    for n in (16, 17, 18, 48, 130):
        d = Decode([n], 4, 4, 2, 128, 16, torch.bfloat16, seed=n)
        want = d.run(P, torch.float32)
        for t in (n - 2, n - 1):
            blk, row = _place(d, 0, t)
            d.vc[blk, :, row] = NAN[0]
        out = d.run(P, torch.float32)
        assert torch.equal(out[0, :2], want[0, :2]) and bool(out[0, 2:].isnan().all())
    assert P.pkv_get_device_error() == 0


@pytest.mark.parametrize("part", [0, 32, 16])
def test_decode_in_pieces_beside_rows_that_nobody_sees(P, part):
    d = Decode([37, 16, 70, 500], 3, 4, 2, 64, 16, torch.float16, seed=5)
    clean = d.run(P, torch.float32, part)
    for s, n in enumerate(d.lens):
        blk = int(d.tables[s, (n - 1) // 16])
        if n % 16:
            d.kc[blk, :, n % 16:] = NAN[0]
            d.vc[blk, :, n % 16:] = NAN[1]
    used = d.tables[d.tables >= 0].long().tolist()
    for b in set(range(d.kc.shape[0])) - set(used):
        d.kc[b], d.vc[b], d.ks[b], d.vs[b] = NAN[0], NAN[0], float("nan"), float("nan")
    assert torch.equal(d.run(P, torch.float32, part), clean)
    assert P.pkv_get_device_error() == 0


def test_decode_of_scales_below_zero(P):
    d = Decode([70, 300, 16], 2, 8, 2, 128, 16, torch.bfloat16, seed=12)
    d.ks[::3] *= -1.0
    d.vs[1::3] *= -1.0
    for out_dtype in (torch.bfloat16, torch.float32):
        d.check(d.run(P, out_dtype))
    assert P.pkv_get_device_error() == 0
