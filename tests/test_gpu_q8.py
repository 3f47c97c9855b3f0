"""The operators on a cache held in 8 bits, on the GPU, against plain models in 64 bits."""
import pytest
import torch

import q8_helpers as Q
import ragged_helpers as R
from gpu_helpers import pkv

pytestmark = pytest.mark.gpu

DEV = "cuda"
DTYPE = R.DTYPE


@pytest.fixture(scope="module")
def P():
    m = pkv()
    m.pkv_get_device_error()
    return m


def _gen(seed):
    return torch.Generator().manual_seed(seed)


# ---------------------------------------------------------------- the write

def _table(max_pos, rot):
    angle = torch.arange(max_pos).double()[:, None] * 10000.0 ** (-torch.arange(0, rot, 2).double() / rot)
    return torch.cat([angle.cos(), angle.sin()], 1).float()


class Write:
    """One call's data: requests (past, new) with their blocks, a cache in use, packed q, k and v."""

    def __init__(self, spans, Hq, Hkv, D, B, dt, seed=0, norm=True, rot=None, interleaved=False, pad=0, size=1.0):
        g = self.g = _gen(seed)
        self.Hq, self.Hkv, self.D, self.B, self.dt = Hq, Hkv, D, B, dt
        lens = [p + n for p, n in spans]
        tables, N = Q.blocks_for(lens, B, g)
        pos, slots = [], []
        for s, (p, n) in enumerate(spans):
            for i in range(p, p + n):
                pos.append(i)
                slots.append(int(tables[s, i // B]) * B + i % B)
        self.tables, self.N = tables, N
        self.pos = torch.tensor(pos + [-1] * pad, dtype=torch.int32)
        self.slots = torch.tensor(slots + [-1] * pad, dtype=torch.int64)
        T = self.T = self.pos.numel()
        self.x = (size * torch.randn(T, (Hq + 2 * Hkv) * D, generator=g)).to(dt)
        self.rot = D if rot is None else rot
        self.cos_sin = _table(max(lens) + 1, self.rot) if self.rot else None
        self.wq, self.wk = ((1 + 0.2 * torch.randn(D, generator=g)).to(dt) if norm else None for _ in range(2))
        self.interleaved, self.eps = interleaved, 1e-5
        (self.kc, self.ks), (self.vc, self.vs) = (Q.random_cache(N, Hkv, B, D, g) for _ in range(2))

    def rows(self, x):
        q, k, v = x.split([self.Hq * self.D, self.Hkv * self.D, self.Hkv * self.D], 1)
        return (t.view(self.T, -1, self.D) for t in (q, k, v))

    def run(self, P, q_out=None, **kw):
        x = self.x.to(DEV)
        q, k, v = self.rows(x)
        self.gpu = [t.to(DEV) for t in (self.kc, self.vc, self.ks, self.vs)]
        self.q_out = torch.full((self.T, self.Hq, self.D), 7.0, dtype=self.dt, device=DEV) if q_out is None else q_out
        up = lambda t: None if t is None else t.to(DEV)  # noqa: E731
        P.pkv_qk_norm_rope_write_q8(q, k, v, *self.gpu, self.pos.to(DEV), self.slots.to(DEV), self.q_out,
                                    q_weight=up(self.wq), k_weight=up(self.wk), eps=self.eps, cos_sin=up(self.cos_sin),
                                    interleaved=self.interleaved, **kw)

    def check(self):
        q, k, v = self.rows(self.x)
        pos = self.pos.long()
        real = pos >= 0
        # q: one rounding of a 32-bit result that is off by a few steps of 2^-24 of its terms
        want, size = R.norm_rope(q[real], self.wq, self.eps, self.cos_sin, pos[real], self.interleaved)
        u = torch.finfo(self.dt).eps / 2
        err = 24 * 2.0 ** -24 * size
        got = self.q_out.cpu()
        off = (got[real].double() - want).abs()
        floor = torch.finfo(self.dt).smallest_normal * u
        assert bool((off <= u * (want.abs() + err) + err + floor).all())
        assert bool((got[~real] == 7).all())
        # k: the code of a number within err of the 64-bit one; v: the code itself
        rows, size = R.norm_rope(k, self.wk, self.eps, self.cos_sin, pos.clamp(min=0), self.interleaved)
        err = 24 * 2.0 ** -24 * size
        for name, x, codes, scale, e, before, before_s in (
                ("k", rows, self.gpu[0], self.gpu[2], err, self.kc, self.ks),
                ("v", v.double(), self.gpu[1], self.gpu[3], torch.zeros_like(err), self.vc, self.vs)):
            host = Q.HostCache(before, before_s)
            places = host.write(x, torch.where(real, self.slots, -1).tolist())
            assert torch.equal(scale.cpu().double(), host.scale), name
            got = codes.cpu().double()
            for t, blk, r in places:
                s = host.scale[blk][:, None]
                g = got[blk, :, r]
                lo, hi = Q.code_of((x[t] - e[t]) / s), Q.code_of((x[t] + e[t]) / s)
                nan = ~torch.isfinite(x[t])
                assert bool(((lo <= g) & (g <= hi) | nan & g.isnan()).all()), (name, t)
                host.codes[blk, :, r] = g
            same = (got == host.codes) | (got.isnan() & host.codes.isnan())
            assert bool(same.all()), name   # every other row: as it was, or rounded to a larger scale


@pytest.mark.parametrize("D,B", [(64, 16), (64, 32), (128, 16), (128, 32)])
@pytest.mark.parametrize("dt,norm,rot,interleaved", [
    ("bf16", True, None, False), ("f16", False, None, True), ("f16", True, 32, False), ("bf16", False, 0, False),
    ("bf16", True, 48, True)])
def test_write_equals_the_plain_model(P, D, B, dt, norm, rot, interleaved):
    # decoding requests at every kind of place, whole prompts, parts that begin and end inside blocks
    spans = [(0, 1), (15, 1), (16, 1), (31, 1), (37, 1), (0, 50), (9, 3), (13, 40), (0, 0), (32, 32), (20, 5)]
    w = Write(spans, 6, 2, D, B, DTYPE[dt], seed=D + B, norm=norm, rot=rot, interleaved=interleaved, pad=3)
    w.run(P)
    w.check()
    assert P.pkv_get_device_error() == 0


@pytest.mark.parametrize("Hq,Hkv,D", [(1, 1, 64), (7, 1, 128), (40, 40, 64), (28, 4, 128), (200, 8, 128), (3, 3, 128),
                                      (96, 96, 128)])
def test_write_of_other_head_counts(P, Hq, Hkv, D):
    w = Write([(3, 1), (0, 37), (16, 17), (5, 2)], Hq, Hkv, D, 16, torch.bfloat16, seed=Hq, pad=1)
    w.run(P)
    w.check()
    assert P.pkv_get_device_error() == 0


@pytest.mark.parametrize("T", [511, 512, 513, 1700])
def test_write_of_many_tokens(P, T):
    w = Write([(0, T - 300), (77, 299), (30, 1)], 8, 2, 128, 16, torch.bfloat16, seed=T)
    w.run(P)
    w.check()
    assert P.pkv_get_device_error() == 0


@pytest.mark.parametrize("Hq,Hkv,D,B", [(4, 2, 64, 16), (4, 2, 64, 32), (8, 2, 128, 16), (5, 5, 128, 32), (12, 12, 64, 16),
                                        (9, 9, 128, 16)])
@pytest.mark.parametrize("dt,norm,rot,interleaved", [("bf16", True, None, False), ("f16", False, 32, True),
                                                     ("bf16", True, 0, False)])
def test_write_of_streamed_tokens(P, Hq, Hkv, D, B, dt, norm, rot, interleaved):
    # whole prompts, parts that begin and end inside blocks, short runs side by side, rows without a token
    spans = [(0, 500), (13, 300), (7, 1), (40, 2), (16, 16), (0, 0), (3, 60)] + [(i % 50, 1 + i % 3) for i in range(120)]
    w = Write(spans, Hq, Hkv, D, B, DTYPE[dt], seed=D + B, norm=norm, rot=rot, interleaved=interleaved, pad=40)
    assert w.T > 1024
    w.run(P)
    w.check()
    assert P.pkv_get_device_error() == 0


def test_write_of_streamed_decoding_requests(P):
    w = Write([(i % 70, 1) for i in range(1100)], 2, 2, 128, 16, torch.bfloat16, seed=1)
    w.run(P)
    w.check()
    assert P.pkv_get_device_error() == 0


def test_write_of_streamed_numbers_that_are_not_finite_and_bad_rows(P):
    w = Write([(0, 700), (5, 400)], 2, 2, 64, 16, torch.float16, seed=2, norm=False, rot=0, size=4.0)
    _, k, v = w.rows(w.x)
    k[3, 0, 5], v[40, 1, 7], v[719, 0, 0] = float("inf"), float("nan"), float("-inf")
    k[64:80, 1] = float("nan")     # a page with nothing finite
    w.run(P)
    w.check()
    assert P.pkv_get_device_error() == 0
    w = Write([(0, 700), (5, 400)], 2, 2, 64, 16, torch.float16, seed=2)
    w.pos[30], w.slots[705] = w.cos_sin.shape[0], w.N * 16
    w.run(P)
    assert P.pkv_get_device_error() == P.DEVERR["POSITION"] | P.DEVERR["SLOT"]
    w.pos[30], w.slots[30], w.slots[705] = -1, -1, -1   # as if there were no token, and no key and value
    w.q_out[30] = 7
    w.check()
    w = Write([(0, 16), (0, 1100)], 2, 1, 64, 16, torch.float16, seed=3)
    w.slots[8:16] = w.slots[0:8].clone()              # a block's first slots a second time
    w.run(P)
    assert P.pkv_get_device_error() == P.DEVERR["SLOT"]
    w.slots[8:16] = -1
    w.check()


@pytest.mark.parametrize("size", [1e-4, 30.0, 300.0])
def test_write_grows_a_page_and_keeps_its_scale(P, size):
    # a page's scale rises with larger numbers, its rows rounded again, and never falls
    w = Write([(5, 1), (17, 4), (30, 20)], 2, 2, 64, 32, torch.float16, seed=3, norm=False, size=size)
    w.run(P)
    w.check()
    again = [t.clone() for t in w.gpu]
    first = (w.kc, w.vc, w.ks, w.vs)
    w.kc, w.vc, w.ks, w.vs = (t.cpu() for t in w.gpu)
    w.run(P)                       # the same tokens once more: nothing is left to change
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(again, w.gpu))
    w.kc, w.vc, w.ks, w.vs = first
    assert P.pkv_get_device_error() == 0


def test_write_that_begins_a_block_forgets_its_scale(P):
    w = Write([(0, 3), (16, 1), (32, 16)], 2, 2, 64, 16, torch.float16, seed=4, norm=False)
    w.ks[:], w.vs[:] = 2.0 ** 40, float("nan")
    w.run(P)
    assert bool((w.gpu[2].cpu()[w.slots // 16] < 1).all()) and bool((w.gpu[3].cpu()[w.slots // 16] < 1).all())
    w.vs[:] = 1.0                  # for the untouched pages of the plain model
    w.gpu[3] = torch.where(w.gpu[3].isnan(), 1.0, w.gpu[3])
    w.check()
    assert P.pkv_get_device_error() == 0


def test_write_of_a_scale_that_is_no_power_of_two(P):
    w = Write([(5, 2), (20, 1), (40, 8)], 2, 2, 64, 16, torch.bfloat16, seed=5, norm=False, rot=0)
    w.vs[:], w.ks[:] = 0.75, 3.0   # larger than the new numbers need: they stay
    w.run(P)
    assert bool((w.gpu[2] == 3.0).all()) and bool((w.gpu[3] == 0.75).all())
    _, k, v = w.rows(w.x)
    for x, codes, s in ((k, w.gpu[0], 3.0), (v, w.gpu[1], 0.75)):
        got = codes.cpu().double()[w.slots // 16, :, w.slots % 16]
        lo, hi = (Q.code_of(x.double() / s * (1 + d * 2.0 ** -22)) for d in (-1, 1))
        assert bool(((got >= torch.minimum(lo, hi)) & (got <= torch.maximum(lo, hi))).all())
    assert P.pkv_get_device_error() == 0


def test_write_of_zeros_tiny_and_infinite_numbers(P):
    w = Write([(0, 4), (16, 16), (33, 1), (48, 2)], 1, 2, 64, 16, torch.bfloat16, seed=6, norm=False, rot=0)
    q, k, v = w.rows(w.x)
    k[0:4], v[0:4] = 0, -0.0                        # a block of zeros: the least scale
    k[4:20] *= 2.0 ** -120                          # below what the least scale holds
    v[5, 0, 3], v[7, 1, 9] = float("inf"), float("nan")
    k[20, 0], v[20, 1] = float("nan"), float("-inf")  # nothing finite: the page keeps its scale
    v[21:] *= 2.0 ** 120
    w.run(P)
    w.check()
    assert bool((w.gpu[2].cpu()[w.slots[0] // 16] == 2.0 ** -100).all())
    assert P.pkv_get_device_error() == 0


def test_write_in_place_of_packed_rows(P):
    w = Write([(0, 21), (6, 1)], 4, 2, 64, 16, torch.float16, seed=7)
    w.run(P)
    want = w.q_out.clone()
    q, k, v = (t.contiguous() for t in w.rows(w.x.to(DEV)))
    caches = [t.to(DEV) for t in (w.kc, w.vc, w.ks, w.vs)]
    P.pkv_qk_norm_rope_write_q8(q, k, v, *caches, w.pos.to(DEV), w.slots.to(DEV), q, q_weight=w.wq.to(DEV),
                                k_weight=w.wk.to(DEV), eps=w.eps, cos_sin=w.cos_sin.to(DEV))
    assert torch.equal(q, want)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(caches, w.gpu))
    assert P.pkv_get_device_error() == 0


def test_write_reports_bad_positions_and_slots(P):
    w = Write([(0, 6), (16, 4), (0, 3)], 2, 2, 64, 16, torch.float16, seed=8)
    good_pos, good_slots = w.pos.clone(), w.slots.clone()
    w.pos[2] = w.cos_sin.shape[0]                    # splits the first run: tokens 3.. go on alone
    w.run(P)
    assert P.pkv_get_device_error() == P.DEVERR["POSITION"]
    w.pos[2], w.slots[2] = -1, -1                    # as if there were no token there
    got, w.q_out[2] = w.q_out.clone(), 7
    w.check()
    assert bool((got[2] == 7).all())
    w.pos, w.slots = good_pos, good_slots.clone()
    w.slots[7] = w.N * 16
    w.run(P)
    assert P.pkv_get_device_error() == P.DEVERR["SLOT"]
    q = w.q_out.clone()
    w.slots[7] = -1                                  # its q is written, its k and v are not
    w.check()
    assert torch.equal(q, w.q_out)


def test_write_refuses_a_block_twice_in_a_row(P):
    # a slot twice, and slots in falling order: the run that comes second is left out
    w = Write([(0, 8)], 2, 2, 64, 16, torch.float16, seed=9)
    base = int(w.slots[0])
    w.slots = torch.tensor([0, 1, 2, 2, 3, 4, 1, 2]) + base
    w.run(P)
    assert P.pkv_get_device_error() == P.DEVERR["SLOT"]
    w.slots = torch.tensor([base, base + 1, base + 2] + [-1] * 5)
    w.check()


@pytest.mark.parametrize("T", [60, 900, 1100])
@pytest.mark.parametrize("B,first,again", [(16, 11, 11), (16, 16, 9), (32, 20, 20), (32, 32, 12)])
@pytest.mark.parametrize("gap", [0, 3])
def test_write_refuses_a_block_that_comes_again_at_once(P, T, B, first, again, gap):
    # a block's first rows, then the same rows again, perhaps behind rows without a token: wherever the
    # rows that are looked at together end, the second run is left out, and what follows is written
    w = Write([(0, T)], 24, 24, 64, B, torch.bfloat16, seed=T + B, norm=False, rot=0)
    base = int(w.slots[0])
    at = first + gap
    w.slots[first:at] = -1
    w.slots[at:at + again] = base + torch.arange(again)
    w.slots[at + again:2 * B + 4] = -1
    w.run(P)
    assert P.pkv_get_device_error() == P.DEVERR["SLOT"]
    w.slots[at:at + again] = -1
    w.check()


def test_write_to_far_blocks_and_on_another_stream(P):
    # places past 2^32 bytes of each pool
    N, Hkv, B, D = 300000, 8, 16, 128
    g = _gen(10)
    pools = [torch.empty(N, Hkv, B, D, dtype=torch.uint8, device=DEV).view(Q.CODE) for _ in range(2)]
    scales = [torch.ones(N, Hkv, device=DEV) for _ in range(2)]
    x = torch.randn(20, Hkv, D, generator=g).to(torch.bfloat16)
    slots = torch.cat([torch.arange(16) + (N - 1) * B, torch.arange(4) + (N - 3) * B])
    q_out = torch.empty(20, Hkv, D, dtype=torch.bfloat16, device=DEV)
    xd, pos, sl = x.to(DEV), torch.arange(20, dtype=torch.int32, device=DEV), slots.to(DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    P.pkv_qk_norm_rope_write_q8(xd, xd, xd, *pools, *scales, pos, sl, q_out, stream=side)
    side.synchronize()
    for pool, scale in zip(pools, scales):
        for blk, rows in ((N - 1, x[:16]), (N - 3, x[16:])):
            host = Q.HostCache(torch.zeros(1, Hkv, B, D), torch.ones(1, Hkv))
            host.write(rows.double(), range(len(rows)))
            assert torch.equal(scale[blk].cpu().double(), host.scale[0])
            assert torch.equal(pool[blk, :, :len(rows)].cpu().double(), host.codes[0, :, :len(rows)])
    assert torch.equal(q_out, xd)
    assert P.pkv_get_device_error() == 0


# ---------------------------------------------------------------- decode

class Decode:
    def __init__(self, lens, NQ, Hq, Hkv, D, B, dt, seed=0, spread=1.0, extra_blocks=0):
        g = self.g = _gen(seed)
        self.lens, self.NQ, self.B, self.dt = lens, NQ, B, dt
        self.tables, N = Q.blocks_for(lens, B, g)
        if extra_blocks:
            self.tables = torch.cat([self.tables, torch.full((len(lens), extra_blocks), -1, dtype=torch.int32)], 1)
        (self.kc, self.ks), (self.vc, self.vs) = (Q.random_cache(N, Hkv, B, D, g, spread) for _ in range(2))
        self.ks *= 0.5 / self.ks.mean()  # scores of a few units; scales that are no powers of two
        self.q = torch.randn(len(lens), NQ, Hq, D, generator=g).to(dt)
        self.scale = D ** -0.5

    def run(self, P, out_dtype=None, part=0, max_ctx=None, stream=None):
        S, NQ, Hq, D = self.q.shape
        mc = max(self.lens) if max_ctx is None else max_ctx
        kc = self.kc.to(DEV)
        ws = P.workspace_tensor(P.pkv_decode_q8_workspace_bytes(kc, S, NQ, Hq, mc, part), DEV).fill_(0xff)
        out = torch.full(self.q.shape, 9.0, dtype=out_dtype or self.dt, device=DEV)
        P.pkv_paged_attention_decode_q8(self.q.to(DEV), kc, self.vc.to(DEV), self.ks.to(DEV), self.vs.to(DEV),
                                        self.tables.to(DEV), torch.tensor(self.lens, dtype=torch.int32, device=DEV),
                                        self.scale, out, mc, part, ws, stream=stream)
        return out.cpu()

    def want(self, lens=None):
        S, NQ, Hq, D = self.q.shape
        k, v = Q.numbers(self.kc, self.ks), Q.numbers(self.vc, self.vs)
        # rows that no query sees may hold anything; the model reads them under a weight of zero
        v = torch.where(torch.isfinite(v), v, 0.0)
        k = torch.where(torch.isfinite(k), k, 0.0)
        starts = [NQ * i for i in range(S + 1)]
        ref, mean, delta, length = R.chunk_attention(self.q.view(S * NQ, Hq, D), k, v, starts, self.tables.clamp(min=0),
                                                     lens or self.lens, self.scale)
        return ref, mean, delta, length, float(v.abs().max())

    def check(self, out, lens=None):
        ref, mean, delta, length, top = self.want(lens)
        p_err = 2.0 ** -22 if out.dtype == torch.float32 else 2.0 ** -11
        tol = Q.attention_tolerance(ref, mean, delta, length, top, p_err, out.dtype)
        off = (out.view(ref.shape).double() - ref).abs()
        assert bool((off <= tol).all()), float((off / tol).max())


@pytest.mark.parametrize("D,B", [(64, 16), (64, 32), (128, 16), (128, 32)])
@pytest.mark.parametrize("Hq,Hkv,NQ", [(4, 4, 1), (8, 2, 1), (7, 1, 1), (16, 1, 1), (12, 6, 3), (8, 1, 5), (40, 2, 2)])
def test_decode_equals_the_plain_model(P, D, B, Hq, Hkv, NQ):
    lens = [1, 5, 15, 16, 17, 31, 33, 64, 100, 129, 400, 0, NQ, 2 * B]
    for dt in (torch.float16, torch.bfloat16):
        d = Decode(lens, NQ, Hq, Hkv, D, B, dt, seed=D + Hq)
        for out_dtype in (dt, torch.float32):
            d.check(d.run(P, out_dtype))
    assert P.pkv_get_device_error() == 0


@pytest.mark.parametrize("Hq,Hkv,NQ,D", [(32, 2, 1, 128), (16, 2, 3, 64), (20, 1, 1, 64)])
def test_decode_of_large_batches_of_many_columns(P, Hq, Hkv, NQ, D):
    # 16 columns a CTA; contexts of one and of several pieces
    lens = [1 + (i * 389) % 700 for i in range(1000)] + [1500]
    d = Decode(lens, NQ, Hq, Hkv, D, 16, torch.bfloat16, seed=Hq)
    d.check(d.run(P))
    d.check(d.run(P, torch.float32, 512))
    d.check(d.run(P, torch.float32, 128))
    assert P.pkv_get_device_error() == 0


@pytest.mark.parametrize("part", [16, 64, 256, 4096, 0])
def test_decode_in_pieces(P, part):
    d = Decode([3000, 1, 0, 511, 512, 513, 2049], 2, 8, 2, 128, 16, torch.bfloat16, seed=part)
    for out_dtype in (torch.bfloat16, torch.float32):
        d.check(d.run(P, out_dtype, part))
    assert P.pkv_get_device_error() == 0


@pytest.mark.parametrize("part", [2 ** 31 - 16, 2 ** 30, 2 ** 28])
@pytest.mark.parametrize("max_ctx", [900, 2 ** 30])
def test_decode_in_pieces_of_any_size(P, part, max_ctx):
    # sums of a position and a piece stay within 32 bits
    d = Decode([900, 1, 0, 333], 2, 8, 2, 128, 16, torch.bfloat16, seed=5)
    d.check(d.run(P, part=part, max_ctx=max_ctx))
    assert P.pkv_get_device_error() == 0


@pytest.mark.parametrize("scale", [-0.1, 0.0, 3.0])
def test_decode_of_other_scales(P, scale):
    d = Decode([40, 300], 1, 4, 2, 64, 16, torch.float16, seed=2)
    d.scale = scale
    d.check(d.run(P, torch.float32))
    assert P.pkv_get_device_error() == 0


def test_decode_of_long_contexts(P):
    d = Decode([40000, 17, 9001], 1, 8, 2, 64, 32, torch.bfloat16, seed=3)
    d.check(d.run(P, torch.float32))
    d.check(d.run(P))
    assert P.pkv_get_device_error() == 0


def test_decode_queries_of_all_sizes(P):
    # rows far from 1, a row of zeros, one large element beside small ones; the scale brings scores back
    d = Decode([90, 200], 4, 2, 1, 128, 16, torch.bfloat16, seed=4)
    big = 2.0 ** torch.tensor([60.0, -60.0, 0.0, 0.0]).view(1, 4, 1, 1)
    d.scale = 2.0 ** -62
    d.q = (d.q * big).to(torch.bfloat16)
    d.q[:, 2] = 0
    d.check(d.run(P, torch.float32))
    d.scale, d.q[:, 3] = 2.0 ** -10, d.q[:, 3] * 2.0 ** -9
    d.q[:, 3, :, 5] = 100.0
    d.q[:, 0] = 1
    d.check(d.run(P, torch.float32))
    assert P.pkv_get_device_error() == 0


def test_decode_rows_that_nobody_sees_may_hold_anything(P):
    d = Decode([37, 16, 70], 3, 4, 2, 64, 16, torch.float16, seed=5)
    clean = d.run(P, torch.float32)
    nan = torch.tensor(float("nan")).to(Q.CODE)
    for s, n in enumerate(d.lens):
        blk = int(d.tables[s, (n - 1) // 16])
        if n % 16:
            d.kc[blk, :, n % 16:] = nan
            d.vc[blk, :, n % 16:] = nan
    used = d.tables[d.tables >= 0].long().tolist()
    for b in set(range(d.kc.shape[0])) - set(used):
        d.kc[b], d.vc[b], d.ks[b], d.vs[b] = nan, nan, float("nan"), float("nan")
    assert torch.equal(d.run(P, torch.float32), clean)
    assert torch.equal(d.run(P, torch.float32, part=32), d.run(P, torch.float32, part=32))
    assert P.pkv_get_device_error() == 0


@pytest.mark.parametrize("part", [0, 16])
def test_decode_values_that_are_not_finite(P, part):
    nan = torch.tensor(float("nan")).to(Q.CODE)
    # a key that is NaN: every row that sees it, of its kv head
    d = Decode([50, 60], 3, 4, 2, 64, 16, torch.bfloat16, seed=6)
    clean = d.run(P, part=part)
    d.kc[int(d.tables[0, 48 // 16]), 0, 48 % 16, 7] = nan
    out = d.run(P, part=part)
    assert bool(out[0, 1:, :2].isnan().all())            # positions 48 and 49 see it, 47 does not
    assert torch.equal(out[0, 0], clean[0, 0]) and torch.equal(out[0, :, 2:], clean[0, :, 2:])
    assert torch.equal(out[1], clean[1])
    # a value that is NaN: its element of the rows that see it
    d = Decode([50, 60], 1, 4, 2, 64, 16, torch.bfloat16, seed=6)
    clean = d.run(P, part=part)
    d.vc[int(d.tables[0, 1]), 1, 3, 9] = nan
    out = d.run(P, part=part)
    assert bool(out[0, :, 2:, 9].isnan().all())
    out[0, :, 2:, 9] = clean[0, :, 2:, 9]
    assert torch.equal(out, clean)
    # queries
    d.vc = torch.where(d.vc.float().isnan(), 0.0, d.vc.float()).to(Q.CODE)
    base = d.run(P, part=part)
    d.q[1, 0, 0, 3], d.q[1, 0, 2, 4] = float("nan"), float("inf")
    out = d.run(P, part=part)
    assert bool(out[1, 0, [0, 2]].isnan().all())
    assert torch.equal(out[0], base[0]) and torch.equal(out[1, 0, [1, 3]], base[1, 0, [1, 3]])
    assert P.pkv_get_device_error() == 0


def test_decode_of_small_weights_and_uneven_scales(P):
    # one token of weight 1 and many of 2^-20 each, whose values are large: their sum counts
    n, D = 20000, 64
    d = Decode([n], 1, 1, 1, D, 16, torch.float16, seed=7)
    d.q[:] = 0
    d.q[..., 0] = 1
    k, v = torch.zeros(d.kc.shape), torch.zeros(d.vc.shape)
    k[..., 0] = -20 * 0.6875                      # about 20 below, in base 2
    v[..., 1] = 448.0
    d.ks[:], d.vs[:] = 1.0, 1.0
    first = int(d.tables[0, 0])
    k[first, :, 0, 0], v[first, :, 0, 0] = 0.0, 1.0
    d.vs[first] = 2.0 ** -9                       # a block of small values beside large ones
    d.kc, d.vc, d.scale = k.to(Q.CODE), v.to(Q.CODE), 1.0
    for out_dtype in (torch.float32, torch.float16):
        d.check(d.run(P, out_dtype))
        d.check(d.run(P, out_dtype, part=512))
    assert P.pkv_get_device_error() == 0


def test_decode_of_pages_whose_scale_is_zero(P):
    d = Decode([64], 1, 4, 2, 64, 16, torch.float16, seed=8)
    d.vs[int(d.tables[0, 2])] = 0.0
    d.ks[int(d.tables[0, 1])] = 0.0
    d.check(d.run(P, torch.float32))
    assert P.pkv_get_device_error() == 0


def test_decode_reports_bad_contexts_and_blocks(P):
    d = Decode([40, 40, 40], 1, 4, 2, 64, 16, torch.float16, seed=9)
    good = d.run(P, torch.float32)
    d.lens = [40, -3, 4000]
    out = d.run(P, torch.float32, max_ctx=40)
    assert P.pkv_get_device_error() == P.DEVERR["CONTEXT"]
    assert torch.equal(out[0], good[0]) and bool((out[1] == 0).all())
    d.lens = [40, 0, 40]
    assert torch.equal(out, d.run(P, torch.float32, max_ctx=40))
    for bad in (-1, d.kc.shape[0], 2 ** 31 - 1):
        d.lens = [40, 40, 40]
        d.tables[1, 1] = bad
        out = d.run(P, torch.float32)
        assert P.pkv_get_device_error() == P.DEVERR["BLOCK_ID"]
        assert torch.equal(out[[0, 2]], good[[0, 2]]) and bool(torch.isfinite(out[1]).all())


def test_decode_of_far_blocks(P):
    # pages past 2^32 bytes
    N, Hkv, B, D = 300000, 8, 16, 128
    g = _gen(11)
    small = Decode([100], 1, 8, 8, D, B, torch.bfloat16, seed=11)
    pools = [torch.empty(N, Hkv, B, D, dtype=torch.uint8, device=DEV).view(Q.CODE) for _ in range(2)]
    scales = [torch.empty(N, Hkv, device=DEV) for _ in range(2)]
    far = torch.randperm(1000, generator=g)[:small.kc.shape[0]] + (N - 1000)
    for pool, scale, codes, s in zip(pools, scales, (small.kc, small.vc), (small.ks, small.vs)):
        pool.view(torch.uint8)[far.to(DEV)] = codes.view(torch.uint8).to(DEV)
        scale[far.to(DEV)] = s.to(DEV)
    tables = far[small.tables.long()].to(torch.int32)
    out = torch.empty(small.q.shape, dtype=torch.bfloat16, device=DEV)
    ws = P.workspace_tensor(P.pkv_decode_q8_workspace_bytes(pools[0], 1, 1, 8, 100), DEV)
    P.pkv_paged_attention_decode_q8(small.q.to(DEV), *pools, *scales, tables.to(DEV),
                                    torch.tensor([100], dtype=torch.int32, device=DEV), small.scale, out, 100, 0, ws)
    assert torch.equal(out.cpu(), small.run(P))
    assert P.pkv_get_device_error() == 0


# ---------------------------------------------------------------- a cache in use

def test_a_step_as_it_is_used(P):
    """Prompts, then decoding, over pools that the calls alone fill: tables and slots from the batch
    building, each step captured once and replayed with the next step's lengths and rows."""
    B, Hq, Hkv, D, S, M, dt = 16, 8, 2, 128, 3, 12, torch.bfloat16
    N = S * M
    g = _gen(12)
    alloc = P.BlockAllocator(N, DEV)
    P.pkv_allocator_reset(alloc)
    i32 = lambda *shape: torch.zeros(*shape, dtype=torch.int32, device=DEV)  # noqa: E731
    tables, past, new = torch.full((S, M), -1, dtype=torch.int32, device=DEV), i32(S), i32(S)
    pools = [torch.zeros(N, Hkv, B, D, dtype=torch.uint8, device=DEV).view(Q.CODE) for _ in range(2)]
    scales = [torch.zeros(N, Hkv, device=DEV) for _ in range(2)]
    cos_sin = _table(M * B, D)
    keys, values = [[] for _ in range(S)], [[] for _ in range(S)]

    class Step:
        def __init__(self, T):
            self.start, self.ctx, self.pos, self.seq, self.status = i32(S + 1), i32(S), i32(T), i32(T), i32(S)
            self.slots = torch.zeros(T, dtype=torch.int64, device=DEV)
            self.x = torch.zeros(T, (Hq + 2 * Hkv) * D, dtype=dt, device=DEV)
            self.q_out = torch.zeros(T, Hq, D, dtype=dt, device=DEV)
            self.out = torch.zeros(T, Hq, D, dtype=torch.float32, device=DEV)
            self.table = cos_sin.to(DEV)
            self.ws = P.workspace_tensor(P.pkv_decode_q8_workspace_bytes(pools[0], S, 1, Hq, M * B), DEV)

        def write(self):
            P.pkv_build_batch(alloc, B, tables, past, new, self.start, self.ctx, self.pos, self.seq, self.slots,
                              self.status)
            q, k, v = (t.view(t.shape[0], -1, D) for t in self.x.split([Hq * D, Hkv * D, Hkv * D], 1))
            P.pkv_qk_norm_rope_write_q8(q, k, v, *pools, *scales, self.pos, self.slots, self.q_out,
                                        cos_sin=self.table)

        def attend(self):
            P.pkv_paged_attention_decode_q8(self.q_out, *pools, *scales, tables, self.ctx, D ** -0.5, self.out, M * B,
                                            workspace=self.ws)

        def remember(self):
            pos, seq = self.pos.cpu().long(), self.seq.cpu()
            _, k, v = (t.view(t.shape[0], -1, D) for t in self.x.cpu().split([Hq * D, Hkv * D, Hkv * D], 1))
            k, _ = R.norm_rope(k, None, 0.0, cos_sin, pos.clamp(min=0), False)
            for t in range(len(seq)):
                if pos[t] >= 0:
                    keys[seq[t]].append(k[t])
                    values[seq[t]].append(v[t].double())

    prompt = Step(70)
    new.copy_(torch.tensor([33, 1, 29], dtype=torch.int32))
    prompt.x.copy_(torch.randn(prompt.x.shape, generator=g))
    prompt.write()
    prompt.remember()
    past.copy_(new)
    new.fill_(1)
    step = Step(S)
    step.x.copy_(torch.randn(step.x.shape, generator=g))
    graph = None
    for n in range(40):
        step.x.copy_(torch.randn(step.x.shape, generator=g) * (1 + n % 7))
        if graph is None:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step.write()
                step.attend()
        graph.replay()
        step.remember()
        past += 1
    assert step.ctx.tolist() == [73, 41, 69]
    k, v = Q.numbers(pools[0], scales[0]), Q.numbers(pools[1], scales[1])
    tab = tables.cpu()
    for s in range(S):
        n = int(step.ctx[s])
        for cache, rows in ((k, keys[s]), (v, values[s])):
            got = cache[tab[s, :R.blocks(n, B)].long()].transpose(1, 2).reshape(-1, Hkv, D)[:n]
            want = torch.stack(rows)
            page = torch.arange(n) // B
            top = torch.stack([want[page == b].abs().amax((0, 2)) for b in range(int(page.max()) + 1)])[page]
            # a number is rounded once, and again each time its page's scale grows (at most 3 times here):
            # half a step each, relative, and half of the least step, 2^-10 of a scale of at most top / 224
            assert bool(((got - want).abs() <= 4 * (want.abs() * 2.0 ** -4 + top[:, :, None] / 224 * 2.0 ** -10)
                         ).all())
    ref, mean, delta, length = R.chunk_attention(step.q_out.cpu(), k, v, [0, 1, 2, 3], tab.clamp(min=0),
                                                 step.ctx.tolist(), D ** -0.5)
    tol = Q.attention_tolerance(ref, mean, delta, length, float(v.abs().max()), 2.0 ** -22, torch.float32)
    assert bool(((step.out.cpu().double() - ref).abs() <= tol).all())
    assert P.pkv_get_device_error() == 0
