"""Attention of ragged chunks over a cache held in 8 bits, on the GPU, against a plain model in 64 bits."""
import pytest
import torch

import q8_helpers as Q
import ragged_helpers as R
from gpu_helpers import pkv

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def P():
    m = pkv()
    m.pkv_get_device_error()
    return m


class Chunk:
    """Requests (past, new) with random blocks, a cache in use and random queries."""

    def __init__(self, spans, Hq, Hkv, D, B, dt, seed=0, room=0):
        g = self.g = torch.Generator().manual_seed(seed)
        self.spans, self.B, self.dt = spans, B, dt
        self.lens = [p + n for p, n in spans]
        self.starts = [0]
        for _, n in spans:
            self.starts.append(self.starts[-1] + n)
        T = self.starts[-1] + room
        self.tables, N = Q.blocks_for(self.lens, B, g)
        (self.kc, self.ks), (self.vc, self.vs) = (Q.random_cache(N, Hkv, B, D, g, 0.4) for _ in range(2))
        self.q = torch.randn(T, Hq, D, generator=g).to(dt)
        self.scale = D ** -0.5

    def run(self, P, out_dtype=None, max_ctx=None):
        T, Hq, D = self.q.shape
        S = len(self.lens)
        mc = max(self.lens) if max_ctx is None else max_ctx
        kc = self.kc.to(DEV)
        ws = P.workspace_tensor(P.pkv_chunk_q8_workspace_bytes(kc, T, S, Hq, mc), DEV).fill_(0xff)
        out = torch.full(self.q.shape, 9.0, dtype=out_dtype or self.dt, device=DEV)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
        P.pkv_paged_attention_chunk_q8(self.q.to(DEV), kc, self.vc.to(DEV), self.ks.to(DEV), self.vs.to(DEV),
                                       i32(self.starts), self.tables.to(DEV), i32(self.lens), self.scale, out, mc, ws)
        return out.cpu()

    def check(self, out, rounded=False):
        k, v = (torch.nan_to_num(Q.numbers(c, s)) for c, s in ((self.kc, self.ks), (self.vc, self.vs)))
        n = self.starts[-1]
        ref, mean, delta, length = R.chunk_attention(self.q, k, v, self.starts, self.tables.clamp(min=0), self.lens,
                                                     self.scale)
        u = 2.0 ** -11    # the products are fp16's, whatever the queries' type
        p_err = u * u if out.dtype == torch.float32 else u
        if rounded:
            # scales that are no powers of two: cached numbers are off by u, relative; so are the
            # values, and each score by u of its terms, twice that on the weights and on l
            p_err = p_err + u + 4 * torch.expm1(u * delta)
        tol = Q.attention_tolerance(ref, mean, delta, length, float(v.abs().max()), p_err, out.dtype)
        off = (out.double() - ref).abs()[:n]
        assert bool((off <= tol[:n]).all()), float((off / tol[:n]).max())
        assert bool((out[n:] == 9).all())


MIXED = [(0, 1), (0, 37), (5, 1), (100, 1), (15, 2), (16, 16), (300, 20), (0, 200), (0, 0), (40, 0), (1, 130),
         (700, 3), (127, 1), (128, 1), (64, 64)]


@pytest.mark.parametrize("D,B", [(64, 16), (64, 32), (128, 16), (128, 32)])
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (8, 2), (7, 1), (12, 6), (28, 4), (16, 1)])
def test_chunk_equals_the_plain_model(P, D, B, Hq, Hkv):
    for dt in (torch.float16, torch.bfloat16):
        c = Chunk(MIXED, Hq, Hkv, D, B, dt, seed=D + Hq, room=3)
        c.check(c.run(P))
        c.check(c.run(P, torch.float32))
    assert P.pkv_get_device_error() == 0


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("spans", [[(0, 1500)], [(3000, 40)], [(2500, 1)], [(0, 700), (900, 300), (33, 1), (1200, 5)],
                                   [(i * 37 % 500, 1) for i in range(400)]])
def test_chunk_of_other_batches(P, spans, dt):
    c = Chunk(spans, 8, 2, 128, 16, dt, seed=len(spans))
    c.check(c.run(P))
    c.check(c.run(P, torch.float32))
    assert P.pkv_get_device_error() == 0


@pytest.mark.parametrize("new", [3, 260])
def test_chunk_of_long_contexts(P, new):
    # pieces longer than what is summed in tensor memory at a time
    c = Chunk([(70000, new)], 2, 1, 64, 32, torch.bfloat16, seed=new)
    c.check(c.run(P))
    assert P.pkv_get_device_error() == 0


def test_chunk_of_scales_that_are_no_powers_of_two(P):
    for dt in (torch.float16, torch.bfloat16):
        c = Chunk(MIXED, 8, 2, 128, 16, dt, seed=3)
        c.ks *= 0.3 + torch.rand(c.ks.shape, generator=c.g)
        c.vs *= 0.3 + torch.rand(c.vs.shape, generator=c.g)
        c.check(c.run(P), rounded=True)
        c.check(c.run(P, torch.float32), rounded=True)
    assert P.pkv_get_device_error() == 0


@pytest.mark.parametrize("power", [-60, -20, 20, 60])
def test_chunk_of_scales_far_from_one(P, power):
    # bf16 has the range; keys small where values are large and the other way round
    c = Chunk(MIXED, 4, 2, 64, 16, torch.bfloat16, seed=4)
    c.ks *= 2.0 ** power
    c.vs *= 2.0 ** -power
    c.scale *= 2.0 ** -power
    c.check(c.run(P))
    c.check(c.run(P, torch.float32))
    assert P.pkv_get_device_error() == 0


def test_chunk_rows_that_nobody_sees_may_hold_anything(P):
    c = Chunk(MIXED, 8, 2, 128, 16, torch.bfloat16, seed=5)
    clean = c.run(P)
    nan = torch.tensor(float("nan")).to(Q.CODE)
    for s, n in enumerate(c.lens):
        if n % 16:
            blk = int(c.tables[s, n // 16])
            c.kc[blk, :, n % 16:] = nan
            c.vc[blk, :, n % 16:] = nan
    used = set(c.tables[c.tables >= 0].long().tolist())
    for b in set(range(c.kc.shape[0])) - used:
        c.kc[b], c.vc[b], c.ks[b], c.vs[b] = nan, nan, float("nan"), float("inf")
    assert torch.equal(c.run(P), clean)
    assert torch.equal(c.run(P), clean)
    assert P.pkv_get_device_error() == 0


def test_chunk_reports_bad_contexts_blocks_and_starts(P):
    c = Chunk([(40, 3), (20, 9), (0, 5)], 4, 2, 64, 16, torch.float16, seed=6)
    good = c.run(P)
    c.lens = [43, 29, 400]
    assert torch.equal(c.run(P, max_ctx=43)[:12], good[:12])
    # the last one is cut to 43 positions, whose second and third table entries are -1
    assert P.pkv_get_device_error() == P.DEVERR["CONTEXT"] | P.DEVERR["BLOCK_ID"]
    c.lens = [43, 29, 5]
    c.tables[1, 0] = c.kc.shape[0] + 5
    out = c.run(P)
    assert P.pkv_get_device_error() == P.DEVERR["BLOCK_ID"]
    assert torch.equal(out[:3], good[:3]) and torch.equal(out[12:], good[12:])
    assert bool(torch.isfinite(out).all())
    c.starts = [0, 12, 3, 17]
    assert bool((c.run(P) == 9).all())
    assert P.pkv_get_device_error() == P.DEVERR["POSITION"]


def test_chunk_and_decode_agree(P):
    # one query a request through both, and drafts
    c = Chunk([(p, 4) for p in (1, 30, 500, 2100)], 8, 2, 128, 16, torch.bfloat16, seed=7)
    a = c.run(P, torch.float32).view(4, 4, 8, 128)
    ws = P.workspace_tensor(P.pkv_decode_q8_workspace_bytes(c.kc, 4, 4, 8, 2104), DEV)
    b = torch.empty(4, 4, 8, 128, device=DEV)
    P.pkv_paged_attention_decode_q8(c.q.view(4, 4, 8, 128).to(DEV), *(t.to(DEV) for t in (c.kc, c.vc, c.ks, c.vs)),
                                    c.tables.to(DEV), torch.tensor(c.lens, dtype=torch.int32, device=DEV), c.scale, b,
                                    2104, 0, ws)
    assert bool(((a - b.cpu()).abs() <= 2.0 ** -12).all())  # both within 2^-14 of sums of numbers below 4
    assert P.pkv_get_device_error() == 0


def test_prompts_as_they_are_used(P):
    """Prompts in two parts through building, write and attention, captured once each and replayed
    with other lengths, against the 64-bit model over the pools that the calls left."""
    B, Hq, Hkv, D, S, M, dt, T = 16, 8, 2, 128, 3, 40, torch.bfloat16, 300
    N = S * M
    g = torch.Generator().manual_seed(8)
    i32 = lambda *shape: torch.zeros(*shape, dtype=torch.int32, device=DEV)  # noqa: E731
    alloc = P.BlockAllocator(N, DEV)
    P.pkv_allocator_reset(alloc)
    tables, past, new = torch.full((S, M), -1, dtype=torch.int32, device=DEV), i32(S), i32(S)
    pools = [torch.zeros(N, Hkv, B, D, dtype=torch.uint8, device=DEV).view(Q.CODE) for _ in range(2)]
    scales = [torch.zeros(N, Hkv, device=DEV) for _ in range(2)]
    angle = torch.arange(M * B).double()[:, None] * 10000.0 ** (-torch.arange(0, D, 2).double() / D)
    table = torch.cat([angle.cos(), angle.sin()], 1).float().to(DEV)
    start, ctx, pos, seq, status = i32(S + 1), i32(S), i32(T), i32(T), i32(S)
    slots = torch.zeros(T, dtype=torch.int64, device=DEV)
    x = torch.zeros(T, (Hq + 2 * Hkv) * D, dtype=dt, device=DEV)
    q_out, out = torch.zeros(T, Hq, D, dtype=dt, device=DEV), torch.zeros(T, Hq, D, device=DEV)
    ws = P.workspace_tensor(P.pkv_chunk_q8_workspace_bytes(pools[0], T, S, Hq, M * B), DEV)

    def step():
        P.pkv_build_batch(alloc, B, tables, past, new, start, ctx, pos, seq, slots, status)
        q, k, v = (t.view(T, -1, D) for t in x.split([Hq * D, Hkv * D, Hkv * D], 1))
        P.pkv_qk_norm_rope_write_q8(q, k, v, *pools, *scales, pos, slots, q_out, cos_sin=table)
        P.pkv_paged_attention_chunk_q8(q_out, *pools, *scales, start, tables, ctx, D ** -0.5, out, M * B, ws)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for news in ([200, 1, 77], [100, 130, 1], [1, 1, 290], [3, 0, 2]):
        new.copy_(torch.tensor(news, dtype=torch.int32))
        x.copy_(torch.randn(x.shape, generator=g))
        graph.replay()
        n = sum(news)
        k, v = Q.numbers(pools[0], scales[0]), Q.numbers(pools[1], scales[1])
        starts = start.tolist()
        assert status.tolist() == [0] * S and starts[-1] == n
        ref, mean, delta, length = R.chunk_attention(q_out.cpu(), k, v, starts, tables.cpu().clamp(min=0),
                                                     ctx.tolist(), D ** -0.5)
        tol = Q.attention_tolerance(ref, mean, delta, length, float(v.abs().max()), 2.0 ** -22, torch.float32)
        assert bool(((out.cpu().double() - ref).abs() <= tol)[:n].all())
        past += new
    assert P.pkv_get_device_error() == 0


@pytest.mark.parametrize("which", ["chunk_q8", "decode_q8", "write_q8", "many_write_q8", "chunk"])
def test_a_call_from_a_thread_that_made_none_before(P, which):
    # once everything that is asked for once is known, a new thread's first call has no context yet
    import threading
    c = Chunk([(0, 1100), (40, 3)], 4, 2, 64, 16, torch.float16, seed=3)
    T, S, mc = c.q.shape[0], 2, max(c.lens)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    q, tables, starts, lens = c.q.to(DEV), c.tables.to(DEV), i32(c.starts), i32(c.lens)
    pools = [t.to(DEV) for t in (c.kc, c.vc, c.ks, c.vs)]
    half = [torch.nan_to_num(Q.numbers(a, b)).half().to(DEV) for a, b in ((c.kc, c.ks), (c.vc, c.vs))]
    out, dec = torch.zeros_like(q), torch.zeros_like(q[:2])
    ws = P.workspace_tensor(max(P.pkv_chunk_q8_workspace_bytes(pools[0], T, S, 4, mc),
                                P.pkv_chunk_workspace_bytes(half[0], T, S, 4, mc)), DEV)
    spare = [torch.zeros_like(t.view(torch.uint8)).view(t.dtype) for t in pools]
    slots = torch.arange(1100, dtype=torch.int64, device=DEV)
    pos, kv, q_out = slots.int(), q[:1100, :2].contiguous(), torch.zeros_like(q[:1100])
    write = lambda n, s: P.pkv_qk_norm_rope_write_q8(q[:n], kv[:n], kv[:n], *spare, pos[:n], slots[:n],  # noqa: E731
                                                     q_out[:n], stream=s)
    call = {"chunk_q8": lambda s: P.pkv_paged_attention_chunk_q8(q, *pools, starts, tables, lens, c.scale, out, mc, ws,
                                                                 stream=s),
            "decode_q8": lambda s: P.pkv_paged_attention_decode_q8(q[:2], *pools, tables, lens, c.scale, dec, mc, 512,
                                                                   None, stream=s),
            "write_q8": lambda s: write(9, s), "many_write_q8": lambda s: write(1100, s),
            "chunk": lambda s: P.pkv_paged_attention_chunk(q, *half, starts, tables, lens, c.scale, out, mc, ws,
                                                           stream=s)}[which]
    stream = torch.cuda.current_stream()
    results = (out, dec, q_out, *spare)
    call(stream)
    want = [t.view(torch.uint8).clone() for t in results]
    assert any(bool(t.any()) for t in want)
    for t in results:
        t.view(torch.uint8).zero_()
    torch.cuda.synchronize()
    failed = []

    def first():
        try:
            call(stream)
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    t = threading.Thread(target=first)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not failed
    assert all(torch.equal(a.view(torch.uint8), b) for a, b in zip(results, want))
    assert P.pkv_get_device_error() == 0


def test_calls_from_several_threads_and_a_graph_beside_them(P):
    # the same calls one after another, from four threads on streams of their own, and replayed from a
    # graph while those run: the same bits each time
    import threading

    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731

    class Work:
        def __init__(self, seed, D, dt):
            c = self.c = Chunk([(0, 150), (700, 1), (33, 40), (1200, 9)], 8, 2, D, 16, dt, seed=seed)
            T, self.S, self.mc = c.q.shape[0], len(c.lens), max(c.lens)
            self.q, self.tables, self.starts, self.lens = c.q.to(DEV), c.tables.to(DEV), i32(c.starts), i32(c.lens)
            self.pools = [t.to(DEV) for t in (c.kc, c.vc, c.ks, c.vs)]
            self.out, self.dec = torch.zeros_like(self.q), torch.zeros_like(self.q[:self.S])
            ws = lambda n: P.workspace_tensor(max(n, 16), DEV)  # noqa: E731
            self.ws = ws(P.pkv_chunk_q8_workspace_bytes(self.pools[0], T, self.S, 8, self.mc))
            self.wd = ws(P.pkv_decode_q8_workspace_bytes(self.pools[0], self.S, 1, 8, self.mc, 64))
            # a write of its own: rows of one request into the first blocks of spare pools
            self.spare = [torch.zeros_like(t.view(torch.uint8)).view(t.dtype) for t in self.pools]
            self.slots = torch.arange(64, dtype=torch.int64, device=DEV)
            self.kv = self.q[:64, :2].contiguous()
            self.q_out = torch.zeros_like(self.q[:64])

        def run(self, stream=None):
            P.pkv_paged_attention_chunk_q8(self.q, *self.pools, self.starts, self.tables, self.lens, self.c.scale,
                                           self.out, self.mc, self.ws, stream=stream)
            P.pkv_paged_attention_decode_q8(self.q[:self.S], *self.pools, self.tables, self.lens, self.c.scale, self.dec,
                                            self.mc, 64, self.wd, stream=stream)
            P.pkv_qk_norm_rope_write_q8(self.q[:64], self.kv, self.kv, *self.spare, self.slots.int(), self.slots,
                                        self.q_out, stream=stream)

        def results(self):
            return [t.view(torch.uint8).clone() for t in (self.out, self.dec, self.q_out, *self.spare)]

        def clear(self):
            for t in (self.out, self.dec, self.q_out, *self.spare):
                t.view(torch.uint8).zero_()

    work = [Work(n, (64, 128)[n % 2], (torch.float16, torch.bfloat16)[n // 2 % 2]) for n in range(5)]
    want = []
    for w in work:
        w.run()
        w.c.check(w.out.cpu())
        want.append(w.results())
        w.clear()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work[4].run()
    torch.cuda.synchronize()
    failed = []

    def loop(w):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(20):
                    w.run()
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=loop, args=(w,)) for w in work[:4]]
    for t in threads:
        t.start()
    for _ in range(20):
        graph.replay()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for w, x in zip(work, want):
        assert all(torch.equal(a, b) for a, b in zip(w.results(), x))
    assert P.pkv_get_device_error() == 0
