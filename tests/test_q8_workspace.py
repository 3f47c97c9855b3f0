"""Sizes of workspaces for decode over a cache held in 8 bits (CPU only: nothing is launched)."""
import ctypes
import os
import shutil

import pytest

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and
                                not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="nvcc not available")


@pytest.fixture(scope="module")
def size():
    from paged_kv_cache_293_gb300 import _build
    _build.build()
    from paged_kv_cache_293_gb300 import pagedkv as P

    def f(S, NQ, Hq, ctx, part=0, Hkv=8, D=128, B=16):
        pool = P.pkv_q8_pool(None, None, None, None, 4, B, Hkv, D)
        return P.lib.pkv_decode_q8_workspace_bytes(ctypes.byref(pool), S, NQ, Hq, ctx, part)
    return f


@pytest.mark.parametrize("Hq,Hkv", [(32, 8), (40, 40), (8, 1), (28, 4)])
@pytest.mark.parametrize("part", [0, 64, 1024])
def test_sizes_grow_with_the_call(size, Hq, Hkv, part):
    # one workspace, made for the largest call, serves the smaller ones
    for ctx in (100, 4097, 8192, 9000, 131072):
        for NQ in (1, 4):
            by_seqs = [size(S, NQ, Hq, ctx, part, Hkv) for S in list(range(1, 200)) + [400, 1000, 5000]]
            assert by_seqs == sorted(by_seqs), (ctx, NQ)
    for S in (1, 8, 30):
        by_ctx = [size(S, 2, Hq, ctx, part, Hkv) for ctx in list(range(1, 20000, 97)) + [1 << 17, 1 << 20]]
        assert by_ctx == sorted(by_ctx), S
        by_queries = [size(S, NQ, Hq, 9000, part, Hkv) for NQ in range(1, 40)]
        assert by_queries == sorted(by_queries), S


def test_sizes_of_short_contexts_and_of_small_batches(size):
    assert size(1000, 4, 32, 4096) == 0
    # eight requests or one of 8192 tokens: the same few results a CTA, far from a row of each 128 tokens
    assert 0 < size(8, 1, 32, 8192) < 2 << 20
    assert size(64, 1, 32, 8192) == size(8, 1, 32, 8192)
