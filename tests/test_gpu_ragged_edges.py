"""The ragged-step operators on the GPU where values, lengths or sizes are extreme, against the
plain models of ragged_helpers.py or results known from the formulas."""
import pytest
import torch

import ragged_helpers as R
from gpu_helpers import pkv
from test_gpu_ragged import DEV, Chunk

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    m = pkv()
    m.pkv_get_device_error()
    return m


# ---------------------------------------------------------------- values that are not finite

# heads, kv heads, contexts, new tokens: every form of piece, with and without a cut context
FORMS = {
    "few_rows": (8, 2, [300, 70], [2, 1]),
    "few_rows_cut": (8, 2, [5000, 70], [1, 1]),
    "one_tile": (4, 4, [300, 200], [70, 90]),
    "one_tile_cut": (4, 1, [5000, 130], [20, 31]),
    "two_tiles": (4, 2, [420, 150], [400, 150]),
    "two_tiles_cut": (4, 4, [2300, 900], [200, 140]),
    "sees_nothing": (4, 2, [5, 40], [9, 3]),
}


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("f32_out", [False, True])
@pytest.mark.parametrize("value", ["nan", "inf", "-inf", "all -inf"])
def test_queries_that_are_not_finite(P, form, f32_out, value):
    """A NaN or an infinity in a query row makes that row NaN, as the formula has it (an infinite
    score less an infinite maximum), whatever piece it falls into; all other rows keep their bits,
    and rows that see nothing are zero."""
    Hq, Hkv, ctx, new = FORMS[form]
    c = Chunk("bf16" if f32_out else "f16", Hq, Hkv, 128, 16, ctx, new, 41, pad=1)
    if value == "all -inf":
        c.dev[1][..., 3].abs_().add_(0.5)       # (unused rows stay NaN)
    out_dtype = torch.float32 if f32_out else None
    ws = c.workspace(P)
    want = c.run(P, out_dtype=out_dtype, ws=ws)
    assert (ws[:8].view(torch.int32)[1].item() > 0) == form.endswith("_cut")   # items that were cut
    hit = torch.zeros(c.T, Hq, dtype=torch.bool)
    for t in sorted({0, new[0] // 2, new[0] - 1, new[0], sum(new) - 1}):
        hit[t, (3 * t + 1) % Hq] = True
    c.dev[0][hit.to(DEV), 3] = float(value.split()[-1])
    got = c.run(P, out_dtype=out_dtype).cpu()
    want = want.cpu()
    sees = torch.cat([torch.arange(n) + k - n + 1 > 0 for k, n in zip(ctx, new)] + [torch.ones(1, dtype=torch.bool)])
    assert torch.equal(got[~hit], want[~hit])
    assert torch.isnan(got[hit & sees[:, None]]).all()
    assert (got[:-1][~sees[:-1]] == 0).all()
    assert P.pkv_get_device_error() == 0


# ---------------------------------------------------------------- where the write's output may lie

@pytest.mark.parametrize("place", ["before", "behind", "in a gap", "one token in place"])
def test_write_output_next_to_its_inputs(P, place):
    """Outputs that touch the packed rows, lie between two rows or are one token's own row: allowed."""
    Hq, Hkv, D, B, T = 4, 2, 64, 16, 1 if place == "one token in place" else 3
    row, n = (Hq + 2 * Hkv) * D, T * Hq * D
    stride = row + n if place == "in a gap" else row
    g = torch.Generator().manual_seed(3)
    buf = torch.randn(2 * n + T * stride, generator=g).to(torch.bfloat16).to(DEV)
    x = buf[n:n + T * stride].view(T, stride)
    q, k, v = (x[:, a * D:b * D].view(T, b - a, D) for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
    at = {"before": 0, "behind": n + T * stride, "in a gap": n + row, "one token in place": n}[place]
    cs = torch.rand(8, D, generator=g).to(DEV)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    slots = torch.arange(T, device=DEV)
    pools = [torch.zeros(1, Hkv, B, D, dtype=torch.bfloat16, device=DEV) for _ in range(4)]
    want = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV)
    P.pkv_qk_norm_rope_write(q, k, v, *pools[:2], pos, slots, want, cos_sin=cs)
    out = buf[at:at + n].view(T, Hq, D)
    P.pkv_qk_norm_rope_write(q, k, v, *pools[2:], pos, slots, out, cos_sin=cs)
    assert torch.equal(out, want) and torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3])
    assert P.pkv_get_device_error() == 0
