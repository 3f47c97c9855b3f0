"""Rules of the ragged-step kernels and entry points that need no GPU to be checked."""
import ctypes
import os
import re
import shutil

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
needs_nvcc = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="nvcc not available")
CSRC = os.path.join(ROOT, "paged_kv_cache_293_gb300", "csrc")


def _code(name):
    """A source file without its comments and with single spaces."""
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    return re.sub(r"\s+", " ", re.sub(r"//[^\n]*", "", text))


def test_every_warpgroup_sets_its_registers_at_one_place():
    """setmaxnreg is undefined where the four warps of a warpgroup do not all take the same one:
    warps 0-7, 8-11 and 12-15 each have one, ahead of the branches that tell their warps apart."""
    body = _code("chunk.cuh").split("chunk_attention_kernel(", 1)[1]
    assert re.findall(r"regs_(?:dec|inc)<(\w+)>\(\);", body) == [
        "CHUNK_REGS_OTHERS", "CHUNK_REGS_OUTPUT", "CHUNK_REGS_SOFTMAX"]
    assert "KV_WARP = 8" in body and "OUT_WARP = 12" in body
    assert "if (warp >= KV_WARP && warp < OUT_WARP) { regs_dec<CHUNK_REGS_OTHERS>();" in body
    assert "} else if (warp >= OUT_WARP) { regs_dec<CHUNK_REGS_OUTPUT>();" in body
    assert "} else { regs_inc<CHUNK_REGS_SOFTMAX>();" in body


@pytest.fixture(scope="module")
def P():
    from paged_kv_cache_293_gb300 import _build
    _build.build()
    from paged_kv_cache_293_gb300 import pagedkv
    return pagedkv


# one packed row a token: 4 q heads, 2 k and 2 v heads of 128, fp16; addresses that nothing reads
T, HQ, HKV, D = 8, 4, 2, 128
ROW = (HQ + 2 * HKV) * D
AT = dict(q=1 << 20, k=(1 << 20) + HQ * D * 2, v=(1 << 20) + (HQ + HKV) * D * 2, wq=1 << 24, wk=1 << 25, cs=1 << 26,
          pos=1 << 27, slot=1 << 28, kp=1 << 32, vp=1 << 33)
OUT = T * HQ * D * 2


def _write(P, out, n=T, stride=ROW, **at):
    a = {**AT, **at}
    pool = P.pkv_pool(a["kp"], a["vp"], 4, 16, HKV, D, 1)
    return P.lib.pkv_qk_norm_rope_write(ctypes.byref(pool), a["q"], stride, a["k"], ROW, a["v"], ROW, n, HQ, a["wq"],
                                        a["wk"], 1e-6, a["cs"], 16, 128, 0, a["pos"], a["slot"], out, None)


@needs_nvcc
@pytest.mark.parametrize("out", [
    AT["q"],                                   # in place, over the other heads of the packed rows
    AT["k"], AT["v"],
    AT["q"] - OUT + 16, AT["q"] + 7 * ROW * 2 + HQ * D * 2 - 16,     # the first and the last 16 bytes of q
    AT["v"] + 7 * ROW * 2 + HKV * D * 2 - 16,                        # the last of v
    AT["wq"], AT["wk"] + D * 2 - 16, AT["cs"] + 16 * 128 * 4 - 16, AT["pos"] + 16, AT["slot"] + 48,
    AT["kp"] + 4 * HKV * 16 * D * 2 - 16, AT["vp"] - 16, AT["vp"]])
def test_write_refuses_an_output_over_its_inputs(P, out):
    """Tokens are read after others have been written, in no fixed order."""
    assert _write(P, out) == P.PKV_ERR_INVALID


@needs_nvcc
def test_write_refuses_an_output_between_unpacked_rows(P):
    """q with rows of its own: packed in place is allowed, shifted or spread rows are not."""
    assert _write(P, 1 << 36, q=1 << 36, stride=HQ * D + 8) == P.PKV_ERR_INVALID
    assert _write(P, (1 << 36) + 16, q=1 << 36, stride=HQ * D) == P.PKV_ERR_INVALID
    assert _write(P, (1 << 36) + HQ * D * 2, q=1 << 36, stride=HQ * D) == P.PKV_ERR_INVALID
    # rows wide apart: the first that the output reaches is not the first row
    assert _write(P, (1 << 36) + 5 * (1 << 16) - 64, q=1 << 36, stride=1 << 15) == P.PKV_ERR_INVALID
    assert _write(P, (1 << 36) - 64, n=1, q=(1 << 36) - 128, stride=0) == P.PKV_ERR_INVALID
