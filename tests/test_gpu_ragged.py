"""The operators of a ragged step on the GPU -- batch building, norms + rotation + cache
write, chunk attention -- against plain models in whole numbers and 64 bits."""
import numpy as np
import pytest
import torch

import ragged_helpers as R
from gpu_helpers import pkv

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def P():
    m = pkv()
    m.pkv_get_device_error()
    return m


def _i32(a):
    return torch.as_tensor(np.ascontiguousarray(a, dtype=np.int32), device=DEV)


# ---------------------------------------------------------------- batch building

class GpuBatch:
    def __init__(self, P, host, max_tokens):
        self.P, self.B = P, host.B
        free = np.full(host.N, -7, np.int32)
        free[:len(host.free)] = host.free
        self.alloc = P.BlockAllocator.of_tensors(_i32(free), _i32([len(host.free)]), _i32(host.refs))
        self.tables = _i32(host.tables)
        S = host.S
        self.out = dict(query_start=_i32(np.full(S + 1, -9)), context=_i32(np.full(S, -9)),
                        positions=_i32(np.full(max_tokens, -9)), token_seq=_i32(np.full(max_tokens, -9)),
                        slots=torch.full((max_tokens,), -9, dtype=torch.int64, device=DEV),
                        status=_i32(np.full(S, -9)))

    def build(self, past, new, **kw):
        o = self.out
        self.P.pkv_build_batch(self.alloc, self.B, self.tables, _i32(past), _i32(new), o["query_start"],
                               o["context"], o["positions"], o["token_seq"], o["slots"], o["status"], **kw)

    def check(self, host, want):
        for k, v in want.items():
            assert self.out[k].tolist() == list(v), k
        assert np.array_equal(self.tables.cpu().numpy(), host.tables)
        assert np.array_equal(self.alloc.refcount.cpu().numpy(), host.refs)
        assert self.alloc.free_count.item() == len(host.free)


def _host_batch(S, past, B, M, spare, seed=0):
    rng = np.random.default_rng(seed)
    held = sum(R.blocks(max(int(p), 0), B) for p in past)
    h = R.HostBatch(held + spare, S, M, B)
    order = rng.permutation(h.N)
    h.free = [int(b) for b in order]
    for s in range(S):
        h.hold(s, max(int(past[s]), 0))
    return h


@pytest.mark.parametrize("S,B,past_max,new_max,spare,room", [
    (1, 16, 1, 1, 4, 0), (1, 32, 0, 5000, 200, 3), (4, 16, 100, 60, 40, 5), (7, 16, 40, 3, 30, 1),
    (1023, 16, 60, 9, 2000, 2), (1025, 32, 200, 40, 4000, 7), (9000, 16, 20, 3, 20000, 11)])
def test_batch_equals_serving_one_by_one(P, S, B, past_max, new_max, spare, room):
    rng = np.random.default_rng(S + B)
    past = rng.integers(0, past_max + 1, S)
    new = rng.integers(0 if S > 1 else new_max, new_max + 1, S)
    M = int(R.blocks(int((past + new).max()), B)) + 1
    h = _host_batch(S, past, B, M, spare)
    T = int(new.sum()) + room
    g = GpuBatch(P, h, T)
    g.build(past, new)
    g.check(h, h.build(past, new, T))
    assert set(g.out["status"].tolist()) == {0}
    assert P.pkv_get_device_error() == 0


def test_batch_statuses(P):
    B, M = 16, 6
    #       fits, invalid, invalid, too long, waits, shared, fits, too many, needs none, after
    past = [20, -1, 5, 90, 33, 24, 16, 30, 17, 48]
    new = [30, 4, -2, 20, 0, 3, 40, 60, 5, 1]
    S = len(past)
    h = _host_batch(S, past, B, M, spare=6)
    h.refs[h.tables[5, 1]] = 2
    T = sum(max(n, 0) for n in new) + 2
    g = GpuBatch(P, h, T)
    g.build(past, new)
    want = h.build(past, new, T)
    assert want["status"] == [0, 2, 2, 2, 0, 3, 0, 1, 0, 1]
    g.check(h, want)
    assert P.pkv_get_device_error() == 0


def test_batch_with_less_room_than_tokens(P):
    past, new = [0, 10, 3], [20, 30, 40]
    h = _host_batch(3, past, 16, 8, spare=20)
    g = GpuBatch(P, h, 45)
    g.build(past, new)
    want = h.build(past, new, 45)
    assert want["status"] == [0, 2, 2] and want["query_start"] == [0, 20, 45, 45]
    g.check(h, want)
    assert P.pkv_get_device_error() == P.DEVERR["POSITION"]


def test_batch_bad_ids_are_reported(P):
    h = _host_batch(2, [20, 0], 16, 4, spare=4)
    g = GpuBatch(P, h, 40)
    g.tables[0, 1] = h.N            # the entry that would receive tokens
    g.build([20, 0], [3, 5])
    assert g.out["status"].tolist() == [2, 0]
    assert g.out["slots"].tolist()[:3] == [-1] * 3
    assert P.pkv_get_device_error() == P.DEVERR["BLOCK_ID"]
    h = _host_batch(1, [0], 16, 4, spare=4)
    g = GpuBatch(P, h, 20)
    g.alloc.free_ids[-1] = -3       # the top of the stack
    g.build([0], [20])
    assert g.tables[0].tolist()[0] == -1 and g.out["slots"].tolist()[:16] == [-1] * 16
    assert P.pkv_get_device_error() == P.DEVERR["BLOCK_ID"]


def test_batch_count_elsewhere_and_no_requests(P):
    h = _host_batch(3, [5, 16, 0], 16, 8, spare=20)
    g = GpuBatch(P, h, 64)
    before = g.alloc.free_count.item()
    left = _i32([0])
    for _ in range(2):              # the same step built twice over the same state
        g.build([5, 16, 0], [30, 1, 17], free_count_out=left)
    assert g.alloc.free_count.item() == before
    want = h.build([5, 16, 0], [30, 1, 17], 64)
    g.alloc.free_count.copy_(left)
    g.check(h, want)
    e = GpuBatch(P, R.HostBatch(8, 0, 4, 16), 5)
    e.build([], [])
    assert e.out["query_start"].tolist() == [0] and e.out["slots"].tolist() == [-1] * 5
    assert e.alloc.free_count.item() == 8
    assert P.pkv_get_device_error() == 0


def test_batch_unaligned_views(P):
    """Token arrays that start off a 16-byte boundary."""
    h = _host_batch(2, [5, 0], 16, 4, spare=8)
    g = GpuBatch(P, h, 40)
    for k in ("positions", "token_seq", "slots"):
        g.out[k] = torch.cat([g.out[k][:1], g.out[k]])[1:]
    g.build([5, 0], [20, 17])
    g.check(h, h.build([5, 0], [20, 17], 40))


# ---------------------------------------------------------------- norms, rotation, cache write

def _rope_case(T, Hq, Hkv, D, B, dtype, norm, rot, pad, max_pos, seed, packed):
    g = torch.Generator().manual_seed(seed)
    dt = R.DTYPE[dtype]
    rows = T + pad
    x = (torch.randn(rows, (Hq + 2 * Hkv) * D, generator=g) * 3).to(dt)
    q, k, v = (t.view(rows, -1, D) for t in x.split([Hq * D, Hkv * D, Hkv * D], 1))
    if not packed:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    N = R.blocks(rows, B) + 2
    slots = torch.randperm(N * B, generator=g)[:rows].clone()
    pos = torch.randint(0, max_pos, (rows,), generator=g, dtype=torch.int32)
    pos[0] = max_pos - 1
    pos[T:] = -1
    if T > 2:
        slots[1] = -1
    cs = None
    if rot:
        ang = torch.arange(max_pos, dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(0, rot, 2, dtype=torch.float64) / rot)
        cs = torch.cat([ang.cos(), ang.sin()], 1).float()
    w = [(1 + 0.3 * torch.randn(D, generator=g)).to(dt) if f else None for f in norm]
    kp = torch.randn(N, Hkv, B, D, generator=g).to(dt)
    return q, k, v, slots, pos, cs, w, kp, kp.flip(0).contiguous()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,Hq,Hkv,D,B,norm,rot,inter,pad,packed", [
    (1, 32, 8, 128, 16, (1, 1), 128, False, 0, True),
    (37, 40, 40, 128, 16, (0, 0), 128, True, 3, False),
    (130, 4, 4, 64, 32, (1, 1), 32, False, 1, True),
    (5, 7, 1, 64, 16, (0, 1), 64, True, 0, True),
    (9, 12, 6, 128, 32, (1, 0), 48, False, 0, True),
    (64, 3, 3, 64, 16, (1, 1), 0, False, 0, True),
    (1500, 16, 4, 64, 16, (1, 1), 64, True, 2, True),
    (3, 70, 1, 128, 16, (1, 1), 96, True, 0, True),
    # enough of them to be streamed
    (2000, 20, 5, 128, 32, (1, 1), 128, False, 5, True),
    (2101, 33, 9, 64, 16, (0, 1), 32, True, 1, True),
    (1500, 21, 21, 128, 16, (1, 0), 0, False, 3, False),
    (900, 52, 3, 128, 16, (1, 1), 128, True, 0, True)])
def test_norm_rope_write(P, dtype, T, Hq, Hkv, D, B, norm, rot, inter, pad, packed):
    q, k, v, slots, pos, cs, w, kp, vp = _rope_case(T, Hq, Hkv, D, B, dtype, norm, rot, pad, 5000,
                                                    T + D, packed)
    dt = R.DTYPE[dtype]
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    if packed:
        x = torch.cat([t.reshape(t.shape[0], -1) for t in (q, k, v)], 1).to(DEV)
        gq, gk, gv = (t.view(t.shape[0], -1, D) for t in x.split([Hq * D, Hkv * D, Hkv * D], 1))
    else:
        gq, gk, gv = dev(q), dev(k), dev(v)
    gkp, gvp = dev(kp), dev(vp)
    out = torch.full((T + pad, Hq, D), 77.0, dtype=dt, device=DEV)
    eps = 1e-5
    P.pkv_qk_norm_rope_write(gq, gk, gv, gkp, gvp, dev(pos), dev(slots), out, q_weight=dev(w[0]),
                             k_weight=dev(w[1]), eps=eps, cos_sin=dev(cs), interleaved=inter)
    assert P.pkv_get_device_error() == 0
    at = pos[:T].long()
    # One rounding to the type (half a step), and in 32 bits: D squares summed and scaled,
    # the reciprocal root, two products and a sum, at most (8 + 4 + 2 + 6) * 2^-24 of the
    # terms' size (a square counts twice in the root and is halved by it)
    def tol(ref, size):
        return torch.finfo(dt).eps / 2 * ref.abs() + 24 * 2.0 ** -24 * size + 2.0 ** -25
    ref, size = R.norm_rope(q[:T], w[0], eps, cs, at, inter)
    got = out.cpu().double()
    assert ((got[:T] - ref).abs() <= tol(ref, size)).all()
    assert (got[T:] == 77.0).all()                   # rows without a token stay as they were
    ref, size = R.norm_rope(k[:T], w[1], eps, cs, at, inter)
    written = slots[:T] >= 0
    wk, wv = kp.clone(), vp.clone()
    sl = slots[:T][written]
    wv[sl // B, :, sl % B] = v[:T][written]
    assert torch.equal(gvp.cpu(), wv)                # a bit copy, and nothing else touched
    got = gkp.cpu()
    assert ((got[sl // B, :, sl % B].double() - ref[written]).abs() <= tol(ref, size)[written]).all()
    wk[sl // B, :, sl % B] = got[sl // B, :, sl % B]
    assert torch.equal(got, wk)


@pytest.mark.parametrize("dtype,T,Hq,Hkv,D,rot", [
    ("f32", 700, 40, 40, 128, 128), ("bf16", 500, 100, 30, 128, 96), ("f16", 1200, 130, 7, 64, 64),
    ("f32", 600, 90, 30, 128, 0), ("bf16", 300, 300, 20, 128, 128)])
def test_norm_rope_write_wide_rows(P, dtype, T, Hq, Hkv, D, rot):
    """Tokens so wide that one or two CTAs' stages fill an SM, or none do."""
    test_norm_rope_write(P, dtype, T, Hq, Hkv, D, 16, (1, rot != 96), rot, rot == 64, 3, True)


@pytest.mark.parametrize("T", [33, 2200])
def test_norm_rope_write_in_place_and_unrotated_infinities(P, T):
    """q_out may be q itself; elements past the rotated ones are not touched by the rotation,
    whatever they hold; a plain copy is exact."""
    Hq, Hkv, D, B = 8, 2, 128, 16
    q, k, v, slots, pos, cs, _, kp, vp = _rope_case(T, Hq, Hkv, D, B, "f16", (0, 0), 64, 0, 300, 3, False)
    q[:, :, 100] = float("inf")
    v[3] = float("nan")
    gq = q.to(DEV)
    other = torch.empty_like(gq)
    gkp, gvp = kp.to(DEV), vp.to(DEV)
    args = (k.to(DEV), v.to(DEV), gkp, gvp, pos.to(DEV), slots.to(DEV))
    P.pkv_qk_norm_rope_write(gq, *args, other, cos_sin=cs.to(DEV))
    P.pkv_qk_norm_rope_write(gq, *args, gq, cos_sin=cs.to(DEV))
    assert torch.equal(gq, other)
    assert torch.equal(gq.cpu()[..., 64:], q[..., 64:])
    assert torch.isfinite(gq[..., :64]).all()
    s3 = int(slots[3])
    assert torch.isnan(gvp[s3 // B, :, s3 % B]).all() and torch.isnan(gvp).sum().item() == Hkv * D


@pytest.mark.parametrize("T,Hq", [(6, 4), (2000, 48)])
def test_norm_rope_write_bad_positions_and_slots(P, T, Hq):
    Hkv, D, B = 2, 64, 16
    q, k, v, slots, pos, cs, _, kp, vp = _rope_case(T, Hq, Hkv, D, B, "bf16", (0, 0), 64, 0, 50, 4, True)
    pos[2] = 50
    slots[3] = kp.shape[0] * B
    slots[1] = -1
    gkp, gvp = kp.to(DEV), vp.to(DEV)
    out = torch.full((T, Hq, D), 5.0, dtype=torch.bfloat16, device=DEV)
    P.pkv_qk_norm_rope_write(q.to(DEV), k.to(DEV), v.to(DEV), gkp, gvp, pos.to(DEV), slots.to(DEV), out,
                             cos_sin=cs.to(DEV))
    assert P.pkv_get_device_error() == P.DEVERR["POSITION"] | P.DEVERR["SLOT"]
    assert (out[2] == 5.0).all() and not (out[3] == 5.0).all()
    changed = (gvp.cpu() != vp).flatten(3).any(-1).transpose(1, 2).reshape(-1, Hkv).any(1).nonzero().flatten()
    assert sorted(changed.tolist()) == sorted(int(slots[i]) for i in [0] + list(range(4, T)))


# ---------------------------------------------------------------- chunk attention

class Chunk:
    """A ragged batch on the host and the device; unused rows of the pools hold NaN."""

    def __init__(self, dtype, Hq, Hkv, D, B, ctx, new, seed, pad=0, width=None, sharpen=None):
        g = torch.Generator().manual_seed(seed)
        self.dt = R.DTYPE[dtype]
        S = len(ctx)
        need = [R.blocks(max(c, 0), B) for c in ctx]
        N = sum(need) + 3
        ids = torch.randperm(N, generator=g).to(torch.int32)
        M = width or max(max(need), 1) + 2
        self.tables = torch.full((S, M), -1, dtype=torch.int32)
        self.k = torch.full((N, Hkv, B, D), float("nan"), dtype=self.dt)
        self.v = torch.full((N, Hkv, B, D), float("nan"), dtype=self.dt)
        at = 0
        for s in range(S):
            for j in range(need[s]):
                b = int(ids[at])
                at += 1
                self.tables[s, j] = b
                n = min(B, ctx[s] - j * B)
                k = torch.randn(Hkv, n, D, generator=g)
                if sharpen is not None:   # scores that keep rising along the context
                    k = k + sharpen * (j * B + torch.arange(n))[None, :, None] / max(ctx)
                self.k[b, :, :n] = k.to(self.dt)
                self.v[b, :, :n] = torch.randn(Hkv, n, D, generator=g).to(self.dt)
        self.start = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32)
        self.ctx = torch.tensor(ctx, dtype=torch.int32)
        T = int(self.start[-1]) + pad
        self.q = torch.randn(T, Hq, D, generator=g)
        if sharpen is not None:
            self.q = self.q + 0.5
        self.q = self.q.to(self.dt)
        self.T, self.pad, self.scale, self.max_ctx = T, pad, D ** -0.5, max(max(ctx), 0)
        self.dev = [t.to(DEV) for t in (self.q, self.k, self.v, self.start, self.tables, self.ctx)]

    def workspace(self, P):
        n = P.pkv_chunk_workspace_bytes(self.dev[1], self.T, len(self.ctx), self.q.shape[1], self.max_ctx)
        return torch.full((n,), 0x7f, dtype=torch.uint8, device=DEV)

    def run(self, P, out_dtype=None, scale=None, out=None, ws=None, **kw):
        q, k, v, start, tables, ctx = self.dev
        if out is None:
            out = torch.full(q.shape, 33.0, dtype=out_dtype or self.dt, device=DEV)
        P.pkv_paged_attention_chunk(q, k, v, start, tables, ctx, self.scale if scale is None else scale, out,
                                    self.max_ctx, self.workspace(P) if ws is None else ws, **kw)
        return out

    def check(self, out, scale=None):
        ref, size, delta, length = R.chunk_attention(self.q, self.k, self.v, self.start, self.tables,
                                                     self.ctx.tolist(), self.scale if scale is None else scale)
        n = self.T - self.pad
        tol = R.chunk_tolerance(ref, size, delta, length, self.dt, out.dtype)
        got = out.cpu()
        assert (got[n:] == 33.0).all()       # rows behind the last request stay as they were
        err = (got.double() - ref).abs()[:n]
        bad = ~(err <= tol[:n])
        assert not bad.any(), "%d of %d values off, first at %s: %.3g > %.3g" % (
            int(bad.sum()), bad.numel(), bad.nonzero()[0].tolist(), float(err[bad][0]), float(tol[:n][bad][0]))


def test_chunk_smallest(P):
    """One token of one request."""
    c = Chunk("bf16", 4, 1, 128, 16, [1], [1], 0)
    c.check(c.run(P))
    assert P.pkv_get_device_error() == 0


@pytest.mark.parametrize("dtype,D,B", [("bf16", 128, 16), ("f16", 128, 32), ("f16", 64, 16), ("bf16", 64, 32)])
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (8, 2), (8, 1), (6, 2), (7, 1), (2, 1), (20, 1)])
def test_chunk_ragged(P, dtype, D, B, Hq, Hkv):
    """Lengths around the tile's and page's edges, requests without queries, without a
    context, and with more queries than positions."""
    ctx = [1, 16, 17, 127, 128, 129, 300, 0, 5, 260, 40, 257]
    new = [1, 1, 17, 127, 3, 129, 70, 4, 9, 0, 33, 257]
    c = Chunk(dtype, Hq, Hkv, D, B, ctx, new, Hq * D + B, pad=3)
    c.check(c.run(P))
    assert P.pkv_get_device_error() == 0


@pytest.mark.parametrize("dtype,Hq,Hkv,D,ctx,new", [
    ("bf16", 8, 2, 128, [1100, 2300, 900], [3, 200, 1]),
    ("f16", 4, 1, 64, [5000], [1]),
    ("f16", 3, 3, 128, [3333, 64], [300, 2]),
    ("bf16", 32, 4, 64, [1536, 7000], [40, 1])])
def test_chunk_long_contexts_are_cut(P, dtype, Hq, Hkv, D, ctx, new):
    """Few rows against long contexts: pieces of the context, merged."""
    c = Chunk(dtype, Hq, Hkv, D, 16, ctx, new, sum(ctx), pad=2)
    out = c.run(P)
    c.check(out)
    assert torch.equal(out, c.run(P))       # and the same bits each time
    assert P.pkv_get_device_error() == 0


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f16", 64)])
@pytest.mark.parametrize("Hq,Hkv", [(3, 3), (4, 1), (16, 1)])
def test_chunk_decoding_requests(P, dtype, D, Hq, Hkv):
    """One query each, contexts around the steps' and their quarters' edges; scores that rise."""
    ctx = [1, 31, 32, 33, 96, 97, 127, 128, 129, 160, 255, 256, 257, 700, 0, 1500]
    c = Chunk(dtype, Hq, Hkv, D, 16, ctx, [1] * len(ctx), 7, pad=1)
    c.check(c.run(P))
    c = Chunk(dtype, Hq, Hkv, D, 32, [900, 2500, 64], [1, 16 // (Hq // Hkv), 1], 8, sharpen=12.0)
    c.check(c.run(P))
    assert P.pkv_get_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
def test_chunk_f32_output(P, dtype, D):
    c = Chunk(dtype, 8, 2, D, 16, [500, 1300, 3], [260, 5, 3], 9, pad=1)
    c.check(c.run(P, out_dtype=torch.float32))


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f16", 64)])
def test_chunk_rising_scores(P, dtype, D):
    """Every step raises the maxima, so the accumulators are rescaled again and again."""
    c = Chunk(dtype, 4, 2, D, 16, [1500, 700], [300, 130], 21, sharpen=12.0)
    c.check(c.run(P))


@pytest.mark.parametrize("scale", [-0.2, 0.0, 1.0, 1e-30])
def test_chunk_scales(P, scale):
    c = Chunk("f16", 4, 2, 128, 16, [400, 31], [150, 31], 5)
    c.check(c.run(P, scale=scale), scale=scale)


@pytest.mark.parametrize("Hq,Hkv", [(64, 1), (128, 1), (66, 2)])
def test_chunk_large_groups(P, Hq, Hkv):
    c = Chunk("bf16", Hq, Hkv, 64, 16, [200, 1, 140, 1100], [7, 1, 140, 1], 5, pad=1)
    c.check(c.run(P))


def test_chunk_many_requests(P):
    rng = np.random.default_rng(3)
    ctx = rng.integers(1, 90, 1500)
    new = np.minimum(ctx, rng.integers(0, 4, 1500))
    c = Chunk("bf16", 2, 1, 64, 16, ctx.tolist(), new.tolist(), 8, pad=1)
    c.check(c.run(P))


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 8, 64), (6, 6, 128), (15, 5, 128)])
def test_chunk_pieces_of_all_kinds_one_after_another(P, Hq, Hkv, D):
    """Many pieces for each CTA, one and two query tiles and all step counts in turn."""
    rng = np.random.default_rng(5)
    ctx, new = [], []
    for i in range(150):
        n = int(rng.choice([1, 2, 5, 16, 17, 64, 65, 130, 200, 257]))
        new.append(n)
        ctx.append(n + int(rng.integers(0, 700)))
    c = Chunk("f16", Hq, Hkv, D, 16, ctx, new, 31, pad=2)
    out = c.run(P)
    c.check(out)
    assert torch.equal(out, c.run(P))
    assert P.pkv_get_device_error() == 0


def test_chunk_agrees_with_decode(P):
    """One query per request: the decode kernel's answer."""
    ctx = [1, 30, 500, 1200, 64]
    c = Chunk("f16", 8, 2, 128, 16, ctx, [1] * 5, 4)
    a = c.run(P, out_dtype=torch.float32)
    q, k, v, _, tables, ctxs = c.dev
    b = torch.empty_like(a)
    ws = P.workspace_tensor(P.pkv_decode_workspace_bytes(k, 5, 8, 1200, 512), DEV)
    P.pkv_paged_attention_decode(q, k, v, tables.clamp(min=0), ctxs, c.scale, b, 1200, 512, ws)
    assert (a - b).abs().max().item() < 2e-5


def test_chunk_device_errors(P):
    c = Chunk("f16", 4, 2, 128, 16, [300, 40], [20, 5], 6)
    c.dev[3][1] = 26                        # past the last token
    out = c.run(P)
    assert P.pkv_get_device_error() == P.DEVERR["POSITION"]
    assert (out == 33.0).all()
    c = Chunk("f16", 4, 2, 128, 16, [300, 40], [20, 5], 6)
    c.dev[4][0, 3] = 99999
    out = c.run(P)
    assert P.pkv_get_device_error() == P.DEVERR["BLOCK_ID"]
    assert torch.isfinite(out).all()
    ref = Chunk("f16", 4, 2, 128, 16, [300, 40], [20, 5], 6).run(P)
    assert torch.equal(out[20:], ref[20:])  # the other request is whole
    c.dev = [t.clone() for t in Chunk("f16", 4, 2, 128, 16, [300, 40], [20, 5], 6).dev]
    c.dev[5][1] = -4
    out = c.run(P)
    assert P.pkv_get_device_error() == P.DEVERR["CONTEXT"]
    assert (out[20:] == 0).all() and torch.equal(out[:20], ref[:20])


def test_chunk_graph_replay_with_new_lengths(P):
    """A captured call takes new lengths, queries and tables in the same buffers."""
    a = Chunk("bf16", 8, 2, 128, 16, [700, 90, 1500], [40, 90, 1], 1, width=100)
    b = Chunk("bf16", 8, 2, 128, 16, [1300, 5, 64], [1, 5, 64], 2, pad=61, width=100)
    T = max(a.T, b.T)
    N = max(a.k.shape[0], b.k.shape[0])
    q = torch.zeros(T, 8, 128, dtype=a.dt, device=DEV)
    k, v = (torch.zeros(N, 2, 16, 128, dtype=a.dt, device=DEV) for _ in range(2))
    start, tables, ctx = (torch.zeros_like(t) for t in a.dev[3:])
    out = torch.zeros_like(q)
    ws = P.workspace_tensor(P.pkv_chunk_workspace_bytes(k, T, 3, 8, 1600), DEV)

    def load(c):
        q[:c.T].copy_(c.dev[0])
        k[:c.k.shape[0]].copy_(c.dev[1])
        v[:c.v.shape[0]].copy_(c.dev[2])
        for x, y in zip((start, tables, ctx), c.dev[3:]):
            x.copy_(y)
        out.fill_(33.0)

    def call():
        P.pkv_paged_attention_chunk(q, k, v, start, tables, ctx, 128 ** -0.5, out, 1600, ws)

    load(a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for c in (b, a, b):
        load(c)
        graph.replay()
        torch.cuda.synchronize()
        c.check(out[:c.T])
    assert P.pkv_get_device_error() == 0


def test_chunk_two_streams(P):
    """Calls at the same time on two streams, each with its own workspace."""
    cs = [Chunk("bf16", 8, 2, 128, 16, [900, 1200], [300, 30], i) for i in (11, 12)]
    want = [c.run(P) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    wss = [c.workspace(P) for c in cs]
    outs = [torch.full_like(w, 33.0) for w in want]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s, ws, o in zip(cs, streams, wss, outs):
            c.run(P, out=o, ws=ws, stream=s)
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert torch.equal(w, o)


# ---------------------------------------------------------------- the three together

@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_ragged_steps_end_to_end(P, dtype):
    """Three steps of an engine: prompts (one in two parts), then everything mixed; tables,
    slots, caches and attention grow together and equal the model's."""
    Hq, Hkv, D, B, S, M = 8, 2, 64, 16, 5, 40
    dt = R.DTYPE[dtype]
    h = R.HostBatch(120, S, M, B)
    steps = [[200, 30, 0, 1, 90], [150, 1, 300, 1, 0], [1, 1, 1, 70, 16]]
    T = max(sum(s) for s in steps) + 4
    g = GpuBatch(P, h, T)
    gen = torch.Generator().manual_seed(17)
    k_pool = torch.full((h.N, Hkv, B, D), float("nan"), dtype=dt, device=DEV)
    v_pool = k_pool.clone()
    ang = torch.arange(700, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)
    cs = torch.cat([ang.cos(), ang.sin()], 1).float().to(DEV)
    w = (1 + 0.1 * torch.randn(D, generator=gen)).to(dt).to(DEV)
    ws = P.workspace_tensor(P.pkv_chunk_workspace_bytes(k_pool, T, S, Hq, M * B), DEV)
    past = np.zeros(S, np.int64)
    for new in steps:
        g.build(past, new)
        want = h.build(past, new, T)
        g.check(h, want)
        n = sum(new)
        x = torch.randn(T, (Hq + 2 * Hkv) * D, generator=gen).to(dt).to(DEV)
        q, k, v = (t.view(T, -1, D) for t in x.split([Hq * D, Hkv * D, Hkv * D], 1))
        q_out = torch.full((T, Hq, D), 2.0, dtype=dt, device=DEV)
        out = torch.full((T, Hq, D), 33.0, dtype=dt, device=DEV)
        o = g.out
        P.pkv_qk_norm_rope_write(q, k, v, k_pool, v_pool, o["positions"], o["slots"], q_out, q_weight=w,
                                 k_weight=w, cos_sin=cs)
        P.pkv_paged_attention_chunk(q_out, k_pool, v_pool, o["query_start"], g.tables, o["context"],
                                    D ** -0.5, out, M * B, ws)
        pos = torch.tensor(want["positions"][:n])
        ref, size = R.norm_rope(k.cpu()[:n], w.cpu(), 1e-6, cs.cpu(), pos, False)
        sl = torch.tensor(want["slots"][:n])
        got = k_pool.cpu()[sl // B, :, sl % B].double()
        assert ((got - ref).abs() <= torch.finfo(dt).eps / 2 * ref.abs() + 24 * 2.0 ** -24 * size + 2.0 ** -25).all()
        ref, size, delta, length = R.chunk_attention(q_out.cpu()[:n], k_pool.cpu(), v_pool.cpu(),
                                                     want["query_start"], torch.as_tensor(h.tables),
                                                     want["context"], D ** -0.5)
        tol = R.chunk_tolerance(ref, size, delta, length, dt, dt)
        assert ((out.cpu()[:n].double() - ref).abs() <= tol).all()
        assert (out[n:] == 33.0).all() and (q_out[n:] == 2.0).all()
        past += np.array(new)
    assert P.pkv_get_device_error() == 0


class Engine:
    """The state of a small engine on the GPU; step() makes the three calls."""

    def __init__(self, P, seed, S=4, T=400, Hq=8, Hkv=2, D=64, B=16, M=40, N=140):
        self.P, self.D, self.B, self.heads = P, D, B, (Hq, Hkv)
        g = torch.Generator().manual_seed(seed)
        dt = torch.bfloat16
        i32 = lambda *n: torch.zeros(*n, dtype=torch.int32, device=DEV)  # noqa: E731
        self.alloc = P.BlockAllocator.of_tensors(torch.randperm(N, generator=g).to(torch.int32).to(DEV),
                                                 _i32([N]), i32(N))
        self.tables, self.past, self.new, self.start, self.ctx = i32(S, M), i32(S), i32(S), i32(S + 1), i32(S)
        self.pos, self.seq, self.status = i32(T), i32(T), i32(S)
        self.slots = torch.zeros(T, dtype=torch.int64, device=DEV)
        self.x = torch.zeros(T, (Hq + 2 * Hkv) * D, dtype=dt, device=DEV)
        self.k_pool = torch.full((N, Hkv, B, D), float("nan"), dtype=dt, device=DEV)
        self.v_pool = self.k_pool.clone()
        self.cs = torch.rand(M * B, D, generator=g).to(DEV)
        self.w = (1 + 0.1 * torch.randn(D, generator=g)).to(dt).to(DEV)
        self.q_out, self.out = (torch.full((T, Hq, D), 7.0, dtype=dt, device=DEV) for _ in range(2))
        self.ws = P.workspace_tensor(P.pkv_chunk_workspace_bytes(self.k_pool, T, S, Hq, M * B), DEV)

    def step(self, **kw):
        (Hq, Hkv), D, T = self.heads, self.D, self.x.shape[0]
        q, k, v = (t.view(T, -1, D) for t in self.x.split([Hq * D, Hkv * D, Hkv * D], 1))
        self.P.pkv_build_batch(self.alloc, self.B, self.tables, self.past, self.new, self.start, self.ctx,
                               self.pos, self.seq, self.slots, self.status, **kw)
        self.P.pkv_qk_norm_rope_write(q, k, v, self.k_pool, self.v_pool, self.pos, self.slots, self.q_out,
                                      q_weight=self.w, k_weight=self.w, cos_sin=self.cs, **kw)
        self.P.pkv_paged_attention_chunk(self.q_out, self.k_pool, self.v_pool, self.start, self.tables,
                                         self.ctx, D ** -0.5, self.out, self.tables.shape[1] * self.B,
                                         self.ws, **kw)

    def bits(self):
        """Everything a step leaves behind."""
        ints = [self.tables, self.start, self.ctx, self.pos, self.seq, self.status, self.slots,
                self.alloc.free_count, self.alloc.refcount]
        return [t.clone() for t in ints] + [t.view(torch.int16).clone()
                                            for t in (self.k_pool, self.v_pool, self.q_out, self.out)]


def _steps(seed, T=400, width=768):
    g = torch.Generator().manual_seed(seed)
    lens = [[200, 30, 0, 1], [0, 1, 300, 1], [1, 1, 1, 70], [1, 1, 1, 1], [1, 0, 1, 1]]
    return [(n, torch.randn(T, width, generator=g).to(torch.bfloat16).to(DEV)) for n in lens]


def test_captured_step_replays_like_eager_steps(P):
    """One graph of the whole step, lengths advancing inside it, for prompts and decoding alike."""
    steps, a, b = _steps(3), Engine(P, 5), Engine(P, 5)
    want = []
    for new, x in steps:
        a.new.copy_(_i32(new))
        a.x.copy_(x)
        a.step()
        a.past += a.new
        want.append(a.bits())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        b.step()
        b.past += b.new
    for (new, x), w in zip(steps, want):
        b.new.copy_(_i32(new))
        b.x.copy_(x)
        graph.replay()
        for u, v in zip(w, b.bits()):
            assert torch.equal(u, v)
    assert P.pkv_get_device_error() == 0


def test_steps_of_two_engines_on_two_streams(P):
    """Two engines' calls at the same time, each on a stream given by name."""
    both = [_steps(8), _steps(9)]
    want = []
    for i, steps in enumerate(both):
        e = Engine(P, 20 + i)
        for new, x in steps:
            e.new.copy_(_i32(new))
            e.x.copy_(x)
            e.step()
            e.past += e.new
        want.append(e.bits())
    engines = [Engine(P, 20 + i) for i in range(2)]
    news = [[_i32(n) for n, _ in steps] for steps in both]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in engines]
    for i in range(len(both[0])):
        for e, steps, new, s in zip(engines, both, news, streams):
            with torch.cuda.stream(s):
                e.new.copy_(new[i])
                e.x.copy_(steps[i][1])
            e.step(stream=s)
            with torch.cuda.stream(s):
                e.past += e.new
    torch.cuda.synchronize()
    for e, w in zip(engines, want):
        for u, v in zip(w, e.bits()):
            assert torch.equal(u, v)
    assert P.pkv_get_device_error() == 0


def test_steps_at_the_far_end_of_a_large_pool(P):
    """Blocks whose offsets pass 2^31 elements: 4.6 GB for K and for V."""
    N, Hq, Hkv, D, B, M = 140000, 32, 4, 128, 32, 50
    new = [1400, 1, 99]
    e = Engine(P, 1, S=3, T=sum(new), Hq=Hq, Hkv=Hkv, D=D, B=B, M=M, N=N)
    e.alloc.free_ids.copy_(torch.arange(N))     # the stack's top is the pool's end
    e.new.copy_(_i32(new))
    e.x.copy_(torch.randn(e.x.shape, generator=torch.Generator().manual_seed(4)))
    e.step()
    ids = torch.arange(N - 60, N)
    tables = e.tables.cpu() - (N - 60)
    used = sum(R.blocks(n, B) for n in new)
    assert e.alloc.free_count.item() == N - used and int(e.tables[0, 0]) == N - 1
    kp, vp = e.k_pool[ids.to(DEV)].cpu(), e.v_pool[ids.to(DEV)].cpu()
    q, k, v = (t.view(sum(new), -1, D) for t in e.x.cpu().split([Hq * D, Hkv * D, Hkv * D], 1))
    at = e.slots.cpu() - (N - 60) * B
    eps = torch.finfo(torch.bfloat16).eps
    for x, got in ((q, e.q_out.cpu()), (k, kp[at // B, :, at % B])):
        ref, size = R.norm_rope(x, e.w.cpu(), 1e-6, e.cs.cpu(), e.pos.cpu().long(), False)
        assert ((got.double() - ref).abs() <= eps / 2 * ref.abs() + 24 * 2.0 ** -24 * size + 2.0 ** -25).all()
    assert torch.equal(vp[at // B, :, at % B], v)
    ref, size, delta, length = R.chunk_attention(e.q_out.cpu(), kp, vp, e.start.tolist(), tables, new, D ** -0.5)
    tol = R.chunk_tolerance(ref, size, delta, length, torch.bfloat16, torch.bfloat16)
    assert ((e.out.cpu().double() - ref).abs() <= tol).all()
    assert P.pkv_get_device_error() == 0


def test_chunk_more_rows_than_32_bits_count(P):
    """2^20 queries of 128 heads: 17 GB of them, and more rows times pieces than 2^31."""
    T, S, G, D, B, n, step = 1 << 20, 64, 128, 64, 32, 1 << 14, 4099
    g = torch.Generator().manual_seed(6)
    base = torch.randn(step, G, D, generator=g).to(torch.bfloat16)
    q = torch.empty(T, G, D, dtype=torch.bfloat16, device=DEV)
    for t in range(0, T, step):
        q[t:t + step].copy_(base[:min(step, T - t)])
    kp, vp = (torch.randn(n // B, 1, B, D, generator=g).to(torch.bfloat16) for _ in range(2))
    tables = torch.randperm(n // B, generator=g).to(torch.int32)[None].repeat(S, 1)  # one context for all
    out = torch.full_like(q, 33.0)
    ws = P.workspace_tensor(P.pkv_chunk_workspace_bytes(kp, T, S, G, n), DEV)
    P.pkv_paged_attention_chunk(q, kp.to(DEV), vp.to(DEV), _i32(np.arange(S + 1) * n), tables.to(DEV),
                                _i32([n] * S), D ** -0.5, out, n, ws)
    assert P.pkv_get_device_error() == 0
    rows = torch.tensor([0, 1, n - 1, n, 7 * n + 130, 40 * n + 9001, T - n, T - 1])
    ref, size, delta, length = R.chunk_attention(base[rows % step], kp, vp, range(len(rows) + 1), tables,
                                                 (rows % n + 1).tolist(), D ** -0.5)
    tol = R.chunk_tolerance(ref, size, delta, length, torch.bfloat16, torch.bfloat16)
    assert ((out[rows.to(DEV)].cpu().double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("new", [[1, 3, 1], [40, 1, 60], [130, 5, 300]])
def test_chunk_rows_between_requests_may_hold_anything(P, new):
    """Query rows of no request hold NaN and infinities, next to those of every form of piece;
    two requests read the same table row."""
    ctx = [n + 150 for n in new]
    c = Chunk("bf16", 8, 2, 128, 16, ctx, new, 12, pad=200)
    want = c.run(P)
    c.dev[0][sum(new):] = float("nan")
    c.dev[0][sum(new) + 1] = float("inf")
    assert torch.equal(c.run(P), want)
    c.check(want)
    d = Chunk("bf16", 8, 2, 128, 16, [ctx[0]] * 2, [new[0]] * 2, 13)
    d.tables[1] = d.tables[0]
    d.dev[4] = d.tables.to(DEV)
    d.check(d.run(P))
    assert P.pkv_get_device_error() == 0


def test_norm_rope_write_streamed_in_a_graph(P):
    """The kernel for many tokens, captured; other positions and slots at the replay."""
    T, Hq, Hkv, D = 2200, 40, 4, 128
    q, k, v, slots, pos, cs, w, kp, vp = _rope_case(T, Hq, Hkv, D, 16, "bf16", (True, True), 64, 0, 3000, 3, True)
    d = [t.to(DEV) for t in (q, k, v, kp, vp, pos, slots)]
    out, want = (torch.zeros(T, Hq, D, dtype=q.dtype, device=DEV) for _ in range(2))
    kw = dict(q_weight=w[0].to(DEV), k_weight=w[1].to(DEV), cos_sin=cs.to(DEV))
    P.pkv_qk_norm_rope_write(*d, out, **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        P.pkv_qk_norm_rope_write(*d, out, **kw)
    d[5].copy_(pos.flip(0))
    d[6].copy_(slots.flip(0))
    eager = [t.clone() for t in d]
    graph.replay()
    P.pkv_qk_norm_rope_write(*eager, want, **kw)
    assert torch.equal(out, want) and not torch.equal(eager[3], kp.to(DEV))
    assert torch.equal(d[3], eager[3]) and torch.equal(d[4], eager[4])
    assert P.pkv_get_device_error() == 0
