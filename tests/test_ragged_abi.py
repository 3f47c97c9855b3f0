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
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    alloc = P.BlockAllocator.of_tensors(i(4), i(1), i(4))
    with pytest.raises(ValueError, match="past_lens"):
        P.pkv_build_batch(alloc, 16, i(2, 4), i(3), i(2), i(3), i(2), i(8), i(8),
                          torch.zeros(8, dtype=torch.int64), i(2))
    with pytest.raises(ValueError, match="slot_mapping"):
        P.pkv_build_batch(alloc, 16, i(2, 4), i(2), i(2), i(3), i(2), i(8), i(8), i(8), i(2))
    with pytest.raises(ValueError, match="current CUDA device"):   # host tensors
        P.pkv_build_batch(alloc, 16, i(2, 4), i(2), i(2), i(3), i(2), i(8), i(8),
                          torch.zeros(8, dtype=torch.int64), i(2))
    with pytest.raises(ValueError):
        P.BlockAllocator.of_tensors(i(4).long(), i(1), i(4))
    h = lambda *s: torch.zeros(s, dtype=torch.float16)  # noqa: E731
    pool = h(4, 2, 16, 64)
    args = (pool, pool, i(3), torch.zeros(3, dtype=torch.int64), h(3, 4, 64))
    with pytest.raises(ValueError, match="packed heads"):
        P.pkv_qk_norm_rope_write(h(4, 3, 64).transpose(0, 1), h(3, 2, 64), h(3, 2, 64), *args)
    with pytest.raises(ValueError, match="k must"):
        P.pkv_qk_norm_rope_write(h(3, 4, 64), h(3, 3, 64), h(3, 2, 64), *args)
    with pytest.raises(ValueError, match="head_dim"):
        P.pkv_qk_norm_rope_write(h(3, 4, 128), h(3, 2, 128), h(3, 2, 128), *args)
    with pytest.raises(ValueError, match="query_start"):
        P.pkv_paged_attention_chunk(h(3, 4, 64), pool, pool, i(2), i(2, 4), i(2), 0.1, h(3, 4, 64), 64,
                                    torch.zeros(1, dtype=torch.uint8))
    with pytest.raises(ValueError, match="q must"):
        P.pkv_paged_attention_chunk(torch.zeros(3, 4, 64), pool, pool, i(3), i(2, 4), i(2), 0.1,
                                    h(3, 4, 64), 64, torch.zeros(1, dtype=torch.uint8))
