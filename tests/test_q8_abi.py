"""Argument checks of the entry points on 8-bit pools, answered before any CUDA call (CPU only)."""
import ctypes
import os
import shutil

import pytest
import torch

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and
                                not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="nvcc not available")

D16 = ctypes.c_void_p(1 << 20)   # a 16-byte aligned stand-in: no call here may dereference it
FAR = ctypes.c_void_p(1 << 30)
ODD = ctypes.c_void_p((1 << 20) + 8)


@pytest.fixture(scope="module")
def P():
    from paged_kv_cache_293_gb300 import _build
    _build.build()
    from paged_kv_cache_293_gb300 import pagedkv
    return pagedkv


def _pool(P, **kw):
    d = dict(k=256, v=65536, k_scale=131072, v_scale=132000, num_blocks=4, block_size=16, num_kv_heads=2, head_dim=128)
    d.update(kw)
    return P.pkv_q8_pool(*(d[n] for n, _ in P.pkv_q8_pool._fields_))


BAD_POOLS = [dict(k=0), dict(v=0), dict(k_scale=0), dict(v_scale=0), dict(k=264), dict(v=65544), dict(k_scale=131074),
             dict(v_scale=132001), dict(num_blocks=0), dict(block_size=0), dict(num_kv_heads=0), dict(head_dim=-1)]


def _write(P, pool=None, dtype=1, T=2, Hq=4, qs=None, ks=256, vs=256, eps=1e-6, cs=D16, maxp=16, rot=128, **p):
    pool = pool if pool is not None else _pool(P)
    g = lambda n: p.get(n, FAR if n == "out" else D16)  # noqa: E731
    return P.lib.pkv_qk_norm_rope_write_q8(ctypes.byref(pool), dtype, g("q"), Hq * 128 if qs is None else qs, g("k"),
                                           ks, g("v"), vs, T, Hq, g("wq"), g("wk"), eps, cs, maxp, rot, 0, g("pos"),
                                           g("slot"), g("out"), None)


def test_write_refusals(P):
    assert _write(P, T=0) == P.PKV_OK
    for bad in BAD_POOLS:
        assert _write(P, pool=_pool(P, **bad)) == P.PKV_ERR_INVALID, bad
    assert _write(P, pool=_pool(P, head_dim=96)) == P.PKV_ERR_UNSUPPORTED
    assert _write(P, pool=_pool(P, block_size=8)) == P.PKV_ERR_UNSUPPORTED
    assert _write(P, dtype=0) == P.PKV_ERR_UNSUPPORTED        # 32-bit rows
    assert _write(P, dtype=3) == P.PKV_ERR_INVALID
    assert _write(P, T=-1) == P.PKV_ERR_INVALID
    assert _write(P, Hq=0) == P.PKV_ERR_INVALID
    assert _write(P, rot=144) == P.PKV_ERR_INVALID
    assert _write(P, rot=24) == P.PKV_ERR_UNSUPPORTED
    assert _write(P, rot=0) == P.PKV_ERR_INVALID              # a table without a rotation
    assert _write(P, cs=None) == P.PKV_ERR_INVALID
    assert _write(P, maxp=0) == P.PKV_ERR_INVALID
    assert _write(P, eps=float("inf")) == P.PKV_ERR_INVALID
    assert _write(P, qs=4 * 128 - 8) == P.PKV_ERR_INVALID     # rows overlap
    assert _write(P, vs=260) == P.PKV_ERR_INVALID             # not whole 16-byte vectors
    for name in ("q", "k", "v", "out", "pos", "slot"):
        assert _write(P, **{name: None}) == P.PKV_ERR_INVALID, name
    for name in ("q", "k", "v", "out", "wq", "wk"):
        assert _write(P, **{name: ODD}) == P.PKV_ERR_INVALID, name


def test_write_refuses_an_output_over_an_input(P):
    at = lambda a: ctypes.c_void_p(a)  # noqa: E731
    # 2 tokens of 4 heads of 128: 2048 bytes
    assert _write(P, q=at(1 << 22), out=at((1 << 22) + 16)) == P.PKV_ERR_INVALID
    for name in ("k", "v", "wq", "wk", "pos", "slot"):
        assert _write(P, **{name: at((1 << 30) + 1024)}) == P.PKV_ERR_INVALID, name
    assert _write(P, cs=at((1 << 30) - 16)) == P.PKV_ERR_INVALID
    # each pool is 16 KB, each array of scales 32 bytes
    for name in ("k", "v", "k_scale", "v_scale"):
        size = 16384 if name in "kv" else 32
        base = getattr(_pool(P), name)
        for out in (base - base % 16 - 2032, base + size - 16 - (base + size) % 16):
            assert _write(P, out=at(max(out, 16))) == P.PKV_ERR_INVALID, (name, out)


def _decode(P, pool=None, dtype=1, NQ=1, S=2, Hq=4, M=4, ctx=64, scale=0.1, out_dtype=1, part=0, ws=None, wsb=0, **p):
    pool = pool if pool is not None else _pool(P)
    g = lambda n: p.get(n, D16)  # noqa: E731
    return P.lib.pkv_paged_attention_decode_q8(ctypes.byref(pool), dtype, g("q"), NQ, S, Hq, g("tables"), M, g("lens"),
                                               ctx, scale, g("out"), out_dtype, part, ws, wsb, None)


def test_write_refuses_arrays_over_one_another(P):
    # the pools end at 256 + 16384 and 65536 + 16384, the scales are 32 bytes each
    for bad in (dict(v=256), dict(v=256 + 16368), dict(k=65536 + 16368), dict(v_scale=131072),
                dict(v_scale=131072 + 28), dict(k_scale=131972), dict(k_scale=256), dict(v_scale=65536 + 16380)):
        assert _write(P, pool=_pool(P, **bad)) == P.PKV_ERR_INVALID, bad


def test_decode_refusals(P):
    assert _decode(P, S=0) == P.PKV_OK
    for bad in BAD_POOLS:
        assert _decode(P, pool=_pool(P, **bad)) == P.PKV_ERR_INVALID, bad
    assert _decode(P, pool=_pool(P, head_dim=32)) == P.PKV_ERR_UNSUPPORTED
    assert _decode(P, dtype=0) == P.PKV_ERR_UNSUPPORTED
    assert _decode(P, dtype=-1) == P.PKV_ERR_INVALID
    assert _decode(P, out_dtype=2) == P.PKV_ERR_UNSUPPORTED   # neither 32-bit nor q's type
    assert _decode(P, Hq=3) == P.PKV_ERR_INVALID              # not shared evenly
    for bad in (dict(NQ=0), dict(S=-1), dict(Hq=0), dict(M=0), dict(ctx=-1), dict(scale=float("nan")), dict(part=-16),
                dict(part=24)):
        assert _decode(P, **bad) == P.PKV_ERR_INVALID, bad
    assert _decode(P, S=65536) == P.PKV_ERR_UNSUPPORTED
    assert _decode(P, ctx=2 ** 30 + 1, part=2 ** 30) == P.PKV_ERR_UNSUPPORTED    # a piece's end passes 32 bits
    assert _decode(P, ctx=2 ** 31 - 1, part=2 ** 20) == P.PKV_ERR_UNSUPPORTED
    assert _decode(P, ctx=16 * 65536, part=16) == P.PKV_ERR_UNSUPPORTED
    assert _decode(P, NQ=2 ** 30, S=2, Hq=4) == P.PKV_ERR_UNSUPPORTED
    for name in ("q", "tables", "lens", "out"):
        assert _decode(P, **{name: None}) == P.PKV_ERR_INVALID, name
    for name in ("q", "out"):
        assert _decode(P, **{name: ODD}) == P.PKV_ERR_INVALID, name


def test_decode_workspace(P):
    size = lambda *a: P.lib.pkv_decode_q8_workspace_bytes(ctypes.byref(_pool(P)), *a)  # noqa: E731
    assert size(2, 1, 4, 64, 64) == 0                         # one piece
    assert size(2, 1, 4, 128, 16) == 0                        # eight, which meet in a cluster
    n = size(2, 1, 4, 129, 16)                                # nine: m, l and 128 numbers a row and piece
    assert n == 2 * 1 * 4 * 9 * (2 + 128) * 4
    assert _decode(P, ctx=129, part=16) == P.PKV_ERR_WORKSPACE
    assert _decode(P, ctx=129, part=16, ws=D16, wsb=n - 1) == P.PKV_ERR_WORKSPACE
    assert _decode(P, ctx=129, part=16, ws=ODD, wsb=n) == P.PKV_ERR_WORKSPACE
    for bad in ((-1, 1, 4, 64, 16), (2, 0, 4, 64, 16), (2, 1, 3, 64, 16), (2, 1, 0, 64, 16), (2, 1, 4, -1, 16),
                (2, 1, 4, 64, -16)):
        assert size(*bad) == 0, bad
    assert P.lib.pkv_decode_q8_workspace_bytes(None, 2, 1, 4, 64, 16) == 0


def _chunk(P, pool=None, dtype=1, T=8, Hq=4, S=2, M=4, ctx=64, scale=0.1, out_dtype=1, ws=D16, wsb=None, **p):
    pool = pool if pool is not None else _pool(P)
    g = lambda n: p.get(n, D16)  # noqa: E731
    if wsb is None:
        wsb = P.lib.pkv_chunk_q8_workspace_bytes(ctypes.byref(pool), T, S, Hq, ctx)
    return P.lib.pkv_paged_attention_chunk_q8(ctypes.byref(pool), dtype, g("q"), T, Hq, g("start"), S, g("tables"), M,
                                              g("lens"), ctx, scale, g("out"), out_dtype, ws, wsb, None)


def test_chunk_refusals(P):
    assert _chunk(P, T=0) == P.PKV_OK and _chunk(P, S=0) == P.PKV_OK
    for bad in BAD_POOLS:
        assert _chunk(P, pool=_pool(P, **bad)) == P.PKV_ERR_INVALID, bad
    assert _chunk(P, pool=_pool(P, block_size=64)) == P.PKV_ERR_UNSUPPORTED
    assert _chunk(P, dtype=0) == P.PKV_ERR_UNSUPPORTED
    assert _chunk(P, out_dtype=2) == P.PKV_ERR_UNSUPPORTED
    assert _chunk(P, Hq=2 * 129) == P.PKV_ERR_UNSUPPORTED     # groups above 128
    assert _chunk(P, pool=_pool(P, num_blocks=1 << 26)) == P.PKV_ERR_UNSUPPORTED
    assert _chunk(P, ctx=(1 << 26) + 1, M=1 << 23) == P.PKV_ERR_UNSUPPORTED
    for bad in (dict(T=-1), dict(S=-1), dict(Hq=0), dict(Hq=3), dict(M=0), dict(ctx=-1), dict(scale=float("inf"))):
        assert _chunk(P, **bad) == P.PKV_ERR_INVALID, bad
    for name in ("q", "start", "tables", "lens", "out"):
        assert _chunk(P, **{name: None}) == P.PKV_ERR_INVALID, name
    for name in ("q", "out"):
        assert _chunk(P, **{name: ODD}) == P.PKV_ERR_INVALID, name
    n = P.lib.pkv_chunk_q8_workspace_bytes(ctypes.byref(_pool(P)), 8, 2, 4, 64)
    assert n > 0 and _chunk(P, wsb=n - 1) == P.PKV_ERR_WORKSPACE
    assert _chunk(P, ws=None) == P.PKV_ERR_WORKSPACE and _chunk(P, ws=ODD) == P.PKV_ERR_WORKSPACE
    assert P.lib.pkv_chunk_q8_workspace_bytes(None, 8, 2, 4, 64) == 0


def test_binding_refusals(P):
    codes, scale = torch.zeros(4, 2, 16, 128, dtype=torch.float8_e4m3fn), torch.zeros(4, 2)
    assert P.make_q8_pool(codes, codes, scale, scale).head_dim == 128
    for bad in ((codes.view(torch.uint8), codes, scale, scale), (codes, codes.view(torch.float8_e5m2), scale, scale),
                (codes, codes[:3], scale, scale), (codes, codes, scale[:, :1], scale), (codes, codes, scale, scale[0]),
                (codes, codes, scale.double(), scale), (codes[0], codes[0], scale, scale),
                (codes.transpose(1, 2), codes.transpose(1, 2), scale, scale), (codes, codes, scale.t(), scale.t())):
        with pytest.raises(ValueError):
            P.make_q8_pool(*bad)
    q = torch.zeros(2, 4, 128, dtype=torch.float16)
    i32 = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):    # not on a CUDA device
        P.pkv_paged_attention_decode_q8(q, codes, codes, scale, scale, i32.view(2, 2), i32[:2], 1.0, q, 16)
    with pytest.raises(ValueError):
        P.pkv_paged_attention_chunk_q8(q, codes, codes, scale, scale, i32[:3], i32.view(2, 2), i32[:2], 1.0, q, 16, i32)
    with pytest.raises(ValueError):
        P.pkv_qk_norm_rope_write_q8(q, q, q, codes, codes, scale, scale, i32[:2], i32[:2].long(), q)
