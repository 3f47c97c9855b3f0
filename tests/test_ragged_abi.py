"""Argument checks of the ragged-step entry points, answered before any CUDA call (CPU only)."""
import ctypes
import os
import shutil

import pytest
import torch

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and
                                not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="nvcc not available")

D16 = ctypes.c_void_p(256)   # a 16-byte aligned stand-in: no call here may dereference it
ODD = ctypes.c_void_p(264)


@pytest.fixture(scope="module")
def P():
    from paged_kv_cache_293_gb300 import _build
    _build.build()
    from paged_kv_cache_293_gb300 import pagedkv
    return pagedkv


def _pool(P, **kw):
    d = dict(k=256, v=512, num_blocks=4, block_size=16, num_kv_heads=2, head_dim=128, dtype=1)
    d.update(kw)
    return P.pkv_pool(*(d[n] for n, _ in P.pkv_pool._fields_))


def _batch(P, B=16, M=4, S=2, T=8, alloc=True, **null):
    a = P.pkv_block_allocator(256, 256, 256, 8 if alloc else 0)
    ptr = lambda n: None if null.get(n) else D16  # noqa: E731
    return P.lib.pkv_build_batch(ctypes.byref(a), B, ptr("tables"), M, ptr("past"), ptr("new"), S, T,
                                 None, ptr("start"), ptr("ctx"), ptr("pos"), ptr("seq"), ptr("slot"),
                                 ptr("status"), None)


def test_build_batch_refusals(P):
    assert _batch(P, B=0) == P.PKV_ERR_INVALID
    assert _batch(P, M=0) == P.PKV_ERR_INVALID
    assert _batch(P, S=-1) == P.PKV_ERR_INVALID
    assert _batch(P, T=-1) == P.PKV_ERR_INVALID
    assert _batch(P, alloc=False) == P.PKV_ERR_INVALID
    for name in ("tables", "past", "new", "start", "ctx", "pos", "seq", "slot", "status"):
        assert _batch(P, **{name: True}) == P.PKV_ERR_INVALID, name


def _rope(P, pool=None, T=2, Hq=4, qs=None, ks=256, vs=256, eps=1e-6, cs=D16, maxp=16, rot=128, **p):
    pool = pool if pool is not None else _pool(P)
    g = lambda n: p.get(n, D16)  # noqa: E731
    return P.lib.pkv_qk_norm_rope_write(ctypes.byref(pool), g("q"), Hq * 128 if qs is None else qs,
                                        g("k"), ks, g("v"), vs, T, Hq, g("wq"), g("wk"), eps, cs, maxp,
                                        rot, 0, g("pos"), g("slot"), g("out"), None)


def test_qk_norm_rope_write_refusals(P):
    assert _rope(P, T=0) == P.PKV_OK
    assert _rope(P, pool=_pool(P, head_dim=96)) == P.PKV_ERR_UNSUPPORTED
    assert _rope(P, T=-1) == P.PKV_ERR_INVALID
    assert _rope(P, Hq=0) == P.PKV_ERR_INVALID
    assert _rope(P, rot=144) == P.PKV_ERR_INVALID             # past the head
    assert _rope(P, rot=24) == P.PKV_ERR_UNSUPPORTED          # not a multiple of 16
    assert _rope(P, rot=0) == P.PKV_ERR_INVALID               # a table without a rotation
    assert _rope(P, cs=None) == P.PKV_ERR_INVALID             # a rotation without a table
    assert _rope(P, maxp=0) == P.PKV_ERR_INVALID
    assert _rope(P, eps=-1.0) == P.PKV_ERR_INVALID
    assert _rope(P, eps=float("nan")) == P.PKV_ERR_INVALID
    assert _rope(P, qs=Hq_less()) == P.PKV_ERR_INVALID        # rows overlap
    assert _rope(P, ks=260) == P.PKV_ERR_INVALID              # not whole 16-byte vectors
    for name in ("q", "k", "v", "out", "pos", "slot"):
        assert _rope(P, **{name: None}) == P.PKV_ERR_INVALID, name
    for name in ("q", "k", "v", "out", "wq", "wk"):
        assert _rope(P, **{name: ODD}) == P.PKV_ERR_INVALID, name


def Hq_less():
    return 4 * 128 - 8


def _chunk(P, pool=None, T=4, Hq=4, S=2, M=4, max_ctx=64, scale=0.1, out_dtype=1, ws=D16,
           ws_bytes=1 << 30, **p):
    pool = pool if pool is not None else _pool(P)
    g = lambda n: p.get(n, D16)  # noqa: E731
    return P.lib.pkv_paged_attention_chunk(ctypes.byref(pool), g("q"), T, Hq, g("start"), S,
                                           g("tables"), M, g("ctx"), max_ctx, scale, g("out"),
                                           out_dtype, ws, ws_bytes, None)


def test_chunk_refusals(P):
    assert _chunk(P, T=0) == P.PKV_OK
    assert _chunk(P, S=0) == P.PKV_OK
    assert _chunk(P, pool=_pool(P, dtype=0), out_dtype=0) == P.PKV_ERR_UNSUPPORTED   # fp32 pool
    assert _chunk(P, out_dtype=2) == P.PKV_ERR_UNSUPPORTED                           # bf16 out, fp16 pool
    assert _chunk(P, Hq=3) == P.PKV_ERR_INVALID
    assert _chunk(P, Hq=2 * 129) == P.PKV_ERR_UNSUPPORTED                            # group of 129
    assert _chunk(P, T=-1) == P.PKV_ERR_INVALID
    assert _chunk(P, S=-1) == P.PKV_ERR_INVALID
    assert _chunk(P, M=0) == P.PKV_ERR_INVALID
    assert _chunk(P, max_ctx=-1) == P.PKV_ERR_INVALID
    assert _chunk(P, scale=float("inf")) == P.PKV_ERR_INVALID
    assert _chunk(P, pool=_pool(P, num_blocks=1 << 26)) == P.PKV_ERR_UNSUPPORTED     # 2^31 rows
    assert _chunk(P, ws=None) == P.PKV_ERR_WORKSPACE
    assert _chunk(P, ws=ODD) == P.PKV_ERR_WORKSPACE
    assert _chunk(P, M=1 << 23, max_ctx=(1 << 26) + 1) == P.PKV_ERR_UNSUPPORTED      # longer contexts
    assert _chunk(P, M=1 << 23, max_ctx=1 << 26, q=None) == P.PKV_ERR_INVALID
    assert _chunk(P, M=4, max_ctx=(1 << 31) - 1, q=None) == P.PKV_ERR_INVALID        # the table bounds it
    need = P.lib.pkv_chunk_workspace_bytes(ctypes.byref(_pool(P)), 4, 2, 4, 64)
    assert need > 0
    assert _chunk(P, ws_bytes=need - 1) == P.PKV_ERR_WORKSPACE
    for name in ("q", "start", "tables", "ctx", "out"):
        assert _chunk(P, **{name: None}) == P.PKV_ERR_INVALID, name
    for name in ("q", "out"):
        assert _chunk(P, **{name: ODD}) == P.PKV_ERR_INVALID, name


def test_chunk_workspace_bytes(P):
    f = lambda *a: P.lib.pkv_chunk_workspace_bytes(ctypes.byref(_pool(P)), *a)  # noqa: E731
    assert f(-1, 1, 4, 64) == 0 and f(1, 1, 3, 64) == 0 and f(1, 1, 4, -1) == 0
    # a short context is never cut: no partial results
    assert f(4, 2, 4, 500) < 8192
    assert f(4, 2, 4, 100000) > f(4, 2, 4, 500)
    # partial results stay bounded, whatever the batch
    assert f(1 << 20, 64, 64, 1 << 20) < 256 << 20


def test_binding_checks_tensors(P):
    """Tensors of a wrong kind, or on the host, are refused before the library is called."""
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    h = lambda *s: torch.zeros(s, dtype=torch.float16)  # noqa: E731
    alloc = P.BlockAllocator.of_tensors(i(4), i(1), i(4))
    slots = torch.zeros(8, dtype=torch.int64)
    pool = h(4, 2, 16, 64)
    with pytest.raises(ValueError):
        P.BlockAllocator.of_tensors(i(4).long(), i(1), i(4))
    with pytest.raises(ValueError, match="current CUDA device"):
        P.pkv_build_batch(alloc, 16, i(2, 4), i(2), i(2), i(3), i(2), i(8), i(8), slots, i(2))
    with pytest.raises(ValueError, match="current CUDA device"):
        P.pkv_qk_norm_rope_write(h(8, 4, 64), h(8, 2, 64), h(8, 2, 64), pool, pool, i(8), slots, h(8, 4, 64))
    with pytest.raises(ValueError, match="current CUDA device"):
        P.pkv_paged_attention_chunk(h(3, 4, 64), pool, pool, i(3), i(2, 4), i(2), 0.1, h(3, 4, 64), 64,
                                    torch.zeros(64, dtype=torch.uint8))


@pytest.mark.parametrize("name,bad", [
    ("past_lens", lambda t: t[:1]), ("query_start", lambda t: t[:2]), ("positions", lambda t: t[:7]),
    ("slot_mapping", lambda t: t.int()), ("slot_mapping", lambda t: t[:7]), ("new_lens", lambda t: t.long()),
    ("context_lens", lambda t: torch.zeros(4, dtype=torch.int32)[::2]), ("seq_status", lambda t: t[:0])])
def test_build_batch_binding_names_the_bad_tensor(P, monkeypatch, name, bad):
    monkeypatch.setattr(P, "_current_device", lambda t, n: -1)  # host tensors pass for the device's
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    args = dict(past_lens=i(2), new_lens=i(2), query_start=i(3), context_lens=i(2), positions=i(8),
                token_seq=i(8), slot_mapping=torch.zeros(8, dtype=torch.int64), seq_status=i(2))
    args[name] = bad(args[name])
    if name == "positions":   # the room is its length: the others disagree with it
        name = "token_seq"
    with pytest.raises(ValueError, match=name):
        P.pkv_build_batch(P.BlockAllocator.of_tensors(i(4), i(1), i(4)), 16, i(2, 4), **args)


def test_rope_and_chunk_bindings_name_the_bad_tensor(P, monkeypatch):
    monkeypatch.setattr(P, "_current_device", lambda t, n: -1)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    h = lambda *s: torch.zeros(s, dtype=torch.float16)  # noqa: E731
    pool, slots, ws = h(4, 2, 16, 64), torch.zeros(3, dtype=torch.int64), torch.zeros(64, dtype=torch.uint8)

    def rope(match, q=h(3, 4, 64), k=h(3, 2, 64), v=h(3, 2, 64), pos=i(3), sl=slots, out=h(3, 4, 64), **kw):
        with pytest.raises(ValueError, match=match):
            P.pkv_qk_norm_rope_write(q, k, v, pool, pool, pos, sl, out, **kw)

    rope("q must", q=h(4, 3, 64).transpose(0, 1))
    rope("k must", k=h(3, 3, 64))
    rope("v must", v=h(3, 2, 64).float())
    rope("head_dim", q=h(3, 4, 128))
    rope("positions", pos=i(2))
    rope("slot_mapping", sl=i(3))
    rope("q_out", out=h(3, 4, 64).float())
    rope("cos_sin", cos_sin=torch.zeros(8, 64, dtype=torch.float64))
    rope("q_weight", q_weight=h(32))
    rope("k_weight", k_weight=torch.ones(64))

    def chunk(match, q=h(3, 4, 64), start=i(3), tables=i(2, 4), ctx=i(2), out=h(3, 4, 64)):
        with pytest.raises(ValueError, match=match):
            P.pkv_paged_attention_chunk(q, pool, pool, start, tables, ctx, 0.1, out, 64, ws)

    chunk("query_start", start=i(2))
    chunk("q must", q=torch.zeros(3, 4, 64))
    chunk("head_dim", q=h(3, 4, 128))
    chunk("out must", out=h(3, 4, 32))
    chunk("block_tables", tables=i(2, 8)[:, :4])
    chunk("context_lens", ctx=i(2).long())
