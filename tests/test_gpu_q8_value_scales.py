"""Chunk attention over a cache held in 8 bits whose pages of values differ in size, on the GPU."""
import pytest
import torch

import q8_helpers as Q
import ragged_helpers as R
from gpu_helpers import pkv
from test_gpu_q8_chunk import Chunk

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def P():
    m = pkv()
    m.pkv_get_device_error()
    return m


def _scale_steps(c, powers, zero):
    """Values of positions 128 i .. 128 i + 127 of each context times 2^powers[i % len(powers)], by their
    pages' scales; elements `zero` are zeros but in pages of the least power."""
    least = min(powers)
    for s, n in enumerate(c.lens):
        for b in range(R.blocks(n, c.B)):
            power = powers[b * c.B // 128 % len(powers)]
            blk = int(c.tables[s, b])
            c.vs[blk] *= 2.0 ** power
            if power > least:
                c.vc[blk, :, :, zero] = torch.tensor(0.0).to(Q.CODE)


def _largest(c, v, elements):
    return float(v[c.tables[c.tables >= 0].long()][..., elements].abs().max())


def _check(c, out, elements):
    """Elements where large pages hold zeros, against a bound that their own values give."""
    k, v = Q.numbers(c.kc, c.ks), Q.numbers(c.vc, c.vs)
    ref, mean, delta, length = R.chunk_attention(c.q, k, v, c.starts, c.tables.clamp(min=0), c.lens, c.scale)
    u = 2.0 ** -11
    p_err = u * u if out.dtype == torch.float32 else u
    ref, mean, out = ref[..., elements], mean[..., elements], out[..., elements]
    tol = Q.attention_tolerance(ref, mean, delta, length, _largest(c, v, elements), p_err, out.dtype)
    off = (out.double() - ref).abs()
    assert bool((off <= tol).all()), float((off / tol).max())


FORMS = [[(900, 3)], [(900, 30)], [(500, 300)], [(0, 700), (300, 1), (1000, 5)], [(5000, 2)], [(4000, 70)]]


@pytest.mark.parametrize("down", [True, False])
@pytest.mark.parametrize("d", [5, 10, 20, 30, 45])
@pytest.mark.parametrize("spans", FORMS)
def test_chunk_of_values_of_two_sizes(P, spans, d, down):
    # few rows, one tile, two tiles, in one piece and cut; the larger step first and last
    for D, dt in ((64, torch.bfloat16), (128, torch.float16)):
        for out_dtype in (torch.float32, dt):
            if dt == torch.float16 and out_dtype == dt and d > 5:
                continue    # fp16 outputs have no room for both
            c = Chunk(spans, 8, 2, D, 16, dt, seed=d)
            elements = torch.arange(3, D, 2)
            _scale_steps(c, [0, -d] if down else [-d, 0], elements)
            out = c.run(P, out_dtype)
            _check(c, out, elements)
            _check(c, out, torch.arange(0, 3))
    assert P.pkv_get_device_error() == 0


def test_chunk_of_values_of_many_sizes(P):
    # up and down by less and by more than fp16 has room for, and pages of zeros with the least scale
    powers = [0, 3, -3, 8, 0, -9, -25, -12, 10, 0, -45, -40, 4, -1]
    for spans in ([(2000, 3)], [(2000, 40)], [(1700, 300)], [(0, 2100)]):
        for D, dt in ((64, torch.float16), (128, torch.bfloat16)):
            c = Chunk(spans, 4, 2, D, 32, dt, seed=D)
            elements = torch.arange(D // 2, D)
            _scale_steps(c, powers, elements)
            for s, n in enumerate(c.lens):
                for b in range(R.blocks(n, c.B)):
                    if b * c.B // 128 % 5 == 2:
                        c.vc[int(c.tables[s, b])] = torch.tensor(0.0).to(Q.CODE)
                        c.vs[int(c.tables[s, b])] = 2.0 ** -100
            out = c.run(P, torch.float32)
            _check(c, out, elements)
            _check(c, out, torch.arange(0, D // 2))
    assert P.pkv_get_device_error() == 0


@pytest.mark.parametrize("new", [2, 20, 140])
@pytest.mark.parametrize("down", [True, False])
def test_chunk_of_long_pieces_of_two_sizes(P, new, down):
    """Contexts of 70000 tokens in one piece each, whose sizes change before, at and after the steps where
    sums go into totals (every 256 steps of 128 tokens)."""
    n, B, D, dt = 70000, 32, 64, torch.bfloat16
    S = 3 * torch.cuda.get_device_properties(0).multi_processor_count + 14
    c = Chunk([(n - new, new)], 1, 1, D, B, dt, seed=new)
    elements = torch.arange(32, 64)
    powers = [0] * 100 + [-20] * 156 + [-18] * 100 + [-40] * 156 + [-5] * 40
    _scale_steps(c, powers if down else [-40 - x for x in powers], elements)
    c.q = torch.randn(S * new, 1, D, generator=c.g).to(dt)
    out = torch.empty(S * new, 1, D, device=DEV)
    kc = c.kc.to(DEV)
    ws = P.workspace_tensor(P.pkv_chunk_q8_workspace_bytes(kc, S * new, S, 1, n), DEV).fill_(0xff)
    P.pkv_paged_attention_chunk_q8(c.q.to(DEV), kc, c.vc.to(DEV), c.ks.to(DEV), c.vs.to(DEV),
                                   torch.arange(0, S * new + 1, new, dtype=torch.int32, device=DEV),
                                   c.tables.repeat(S, 1).to(DEV), torch.full((S,), n, dtype=torch.int32, device=DEV),
                                   c.scale, out, n, ws)
    assert P.pkv_get_device_error() == 0
    assert ws[:8].view(torch.int32)[1].item() == 0     # none was cut
    some = [0, 151, S - 1]
    rows = torch.cat([torch.arange(s * new, (s + 1) * new) for s in some])
    k, v = Q.numbers(c.kc, c.ks), Q.numbers(c.vc, c.vs)
    ref, mean, delta, length = R.chunk_attention(c.q[rows], k, v, range(0, len(rows) + 1, new), c.tables.repeat(3, 1),
                                                 [n] * 3, c.scale)
    for e in (elements, torch.arange(0, 32)):
        # (sums count 2^-23 a token over 2^15 tokens at most, and three totals)
        tol = Q.attention_tolerance(ref[..., e], mean[..., e], delta, length.clamp(max=2 ** 15 + 3),
                                    _largest(c, v, e), 2.0 ** -22, torch.float32)
        tol = tol + n * 2.0 ** -32 * _largest(c, v, e)
        off = (out[rows.to(DEV)].cpu().double() - ref)[..., e].abs()
        assert bool((off <= tol).all()), float((off / tol).max())


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
def test_chunk_of_scales_of_zero_and_below(P, dt):
    # pages of scale zero alone in a step and beside others, and scales that turn the sign
    c = Chunk([(0, 300), (700, 3), (130, 40), (513, 1)], 8, 2, 128, 16, dt, seed=9)
    for s, n in enumerate(c.lens):
        for b in range(R.blocks(n, c.B)):
            blk = int(c.tables[s, b])
            if b // 8 % 3 == 1 or b % 5 == 2:
                c.vs[blk] = 0.0
            if b % 7 == 3:
                c.ks[blk] = 0.0
            if b % 4 == 1:
                c.vs[blk, 0] *= -1.0
                c.ks[blk, 1] *= -1.0
    for out_dtype in (dt, torch.float32):
        c.check(c.run(P, out_dtype))
    assert P.pkv_get_device_error() == 0


def test_chunk_of_values_of_many_sizes_gives_the_same_bits(P):
    # whichever CTA takes a piece, and whatever it had before: also with scales that are no powers of two
    spans = [(i * 97 % 900, 1 + i % 3) for i in range(300)] + [(i * 331 % 2000, 20 + i * 7 % 200) for i in range(12)]
    for dt, odd in ((torch.float16, False), (torch.bfloat16, True)):
        c = Chunk(spans, 8, 2, 64, 16, dt, seed=11)
        power = torch.randint(-30, 20, (c.vs.shape[0], 1), generator=c.g)
        c.vs *= torch.pow(2.0, power.float())
        if odd:
            c.vs *= 0.5 + torch.rand(c.vs.shape, generator=c.g)
        want = c.run(P)
        for _ in range(5):
            assert torch.equal(c.run(P), want)
    assert P.pkv_get_device_error() == 0
