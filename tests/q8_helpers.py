"""Plain 64-bit models of the operators on a cache held in 8 bits, for the GPU tests."""
import torch

import ragged_helpers as R

CODE = torch.float8_e4m3fn


def code_of(x):
    """x (64 bits) at the nearest e4m3 value, even at ties: 4 significant bits, steps of 2^-9 at
    least, 448 at most; NaN where x is not finite."""
    _, e = torch.frexp(x)
    step = torch.pow(2.0, (e - 4).clamp(min=-9).double())
    c = (torch.round(x / step) * step).clamp(-448, 448)
    return torch.where(torch.isfinite(x), c, float("nan"))


def scale_for(top):
    """The least power of two, 2^-100 at least, whose 448 times reach top."""
    p = -100
    while top > 448.0 * 2.0 ** p:
        p += 1
    return 2.0 ** p


class HostCache:
    """Keys (or values) of a cache in 8 bits: values of the codes and scales, in 64 bits, on the CPU."""

    def __init__(self, codes, scale):
        self.codes, self.scale = codes.cpu().double(), scale.cpu().double()

    def write(self, x, slots):
        """Rows x [T][Hkv][D] (64 bits) at slots (-1: none), run by run (slots of one block that
        advance as their rows do); returns the places written."""
        B, T = self.codes.shape[2], x.shape[0]
        places, done = [], set()
        for t in range(T):
            s = int(slots[t])
            if s < 0 or t in done:
                continue
            blk, r0, run = s // B, s % B, []
            for i in range(t, T):
                if int(slots[i]) < 0:
                    continue
                if int(slots[i]) != s + i - t or int(slots[i]) // B != blk:
                    break
                run.append(i)
            done.update(run)
            at = torch.tensor([r0 + i - t for i in run])
            for h in range(x.shape[1]):
                rows = x[run, h]
                fine = rows[torch.isfinite(rows)].abs()
                new = scale_for(float(fine.max()) if fine.numel() else 0.0)
                old = float(self.scale[blk, h])
                if r0 > 0:
                    new = max(old, new)
                    if new > old:
                        self.codes[blk, h] = code_of(self.codes[blk, h] * (old / new))
                self.scale[blk, h] = new
                self.codes[blk, h, at] = code_of(rows / new)
            places += [(i, blk, r0 + i - t) for i in run]
        return places


def random_cache(N, Hkv, B, D, g, spread=1.0):
    """(codes, scale) of a pool in use: random numbers whose pages differ in size, by the least scales."""
    x = torch.randn(N, Hkv, B, D, generator=g) * torch.exp(spread * torch.randn(N, Hkv, 1, 1, generator=g))
    top = x.abs().amax((2, 3))
    p = torch.ceil(torch.log2(top.double() / 448))
    scale = torch.pow(2.0, p).float()
    return (x / scale[:, :, None, None]).to(CODE), scale


def numbers(codes, scale):
    """What a pool's values stand for, in 64 bits, on the CPU."""
    return codes.cpu().double() * scale.cpu().double()[:, :, None, None]


def attention_tolerance(ref, mean_abs, delta, length, largest_v, p_err, out_dtype):
    """Largest |error| of an attention output over 8-bit pools, from the roundings it goes through.

    The cached numbers and queries enter exactly.  p_err: what rounding a weight for its product
    does, relative, so p_err * A with A = sum p_i |v_i| / l; fp16 weights are besides off by at most
    2^-32 of the row's largest, which l is no less than: length * 2^-32 * largest |v|.  Scores:
    D-term products summed in 32 bits, at most 128 * 2^-23 * terms off (the tensor cores may
    truncate: one whole step an addition), and four roundings of a scaled score (page and row
    factors, their product, base 2); twice that, relative, on the weights and again on l.  Sums over
    `length` tokens in 32 bits: length * 2^-23 relative to A, for O and for l.  2^-20 for the
    exponentials, the rescalings and divisions.  Last, half a step of the output's type."""
    u_out = torch.finfo(out_dtype).eps / 2
    d = delta * (128 * 2.0 ** -23 + 4 * 2.0 ** -23)
    tol = mean_abs * (p_err + 2 * torch.expm1(d) + 2 * length * 2.0 ** -23 + 2.0 ** -20)
    tol = tol + length * 2.0 ** -32 * largest_v
    return (tol + u_out * (ref.abs() + tol)) * (1 + 1e-6) + 1e-30


def blocks_for(lens, B, g, spare=3):
    """(block tables, pool size): random blocks for each context, -1 past its own."""
    need = [R.blocks(n, B) for n in lens]
    N = sum(need) + spare
    ids = torch.randperm(N, generator=g).to(torch.int32)
    M = max(max(need), 1)
    tables = torch.full((len(lens), M), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        tables[s, :n] = ids[at:at + n]
        at += n
    return tables, N
