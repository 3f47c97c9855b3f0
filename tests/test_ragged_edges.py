"""Rules of the ragged-step kernels and entry points that need no GPU to be checked."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
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
