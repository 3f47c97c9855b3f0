"""Plain models of the ragged-step operators, in whole numbers and 64 bits, for the GPU tests."""
import numpy as np
import torch

DTYPE = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def blocks(n, B):
    return -(-n // B)


class HostBatch:
    """The serving of requests one by one: a free stack popped from its end."""

    def __init__(self, num_blocks, S, M, B):
        self.N, self.S, self.M, self.B = num_blocks, S, M, B
        self.free = list(range(num_blocks - 1, -1, -1))
        self.refs = np.zeros(num_blocks, np.int32)
        self.tables = np.full((S, M), -1, np.int32)

    def hold(self, s, tokens):
        """Row s holds `tokens` tokens in blocks popped now."""
        for j in range(blocks(tokens, self.B)):
            b = self.free.pop()
            self.tables[s, j] = b
            self.refs[b] = 1

    def build(self, past, new, max_tokens):
        B, free, end, upto = self.B, len(self.free), 0, 0
        out = dict(query_start=[0], context=[], positions=[], token_seq=[], slots=[], status=[])
        served = []
        for s in range(self.S):
            p, n = int(past[s]), int(new[s])
            status, need = 0, 0
            if p < 0 or n < 0 or p + n > self.M * B:
                status = 2
            elif n > 0 and p % B and not 0 <= self.tables[s, p // B] < self.N:
                status = 2
            elif n > 0 and p % B and self.refs[self.tables[s, p // B]] != 1:
                status = 3
            elif n > 0:
                need = blocks(p + n, B) - blocks(p, B)
            end += max(n, 0)
            upto += need
            if n > 0 and end > max_tokens:
                status = 2
            elif status == 0 and need and upto > free:
                status = 1
            served.append((need, upto))
            out["query_start"].append(min(end, max_tokens))
            out["status"].append(status)
            out["context"].append(p + n if status == 0 else 0)
        last = 0
        for s in range(self.S):
            need, u = served[s]
            if out["status"][s] == 0 and need:
                for j in range(need):
                    b = self.free[free - 1 - (u - need + j)]
                    self.tables[s, blocks(int(past[s]), B) + j] = b
                    self.refs[b] = 1
                last = u
            for i in range(out["query_start"][s], out["query_start"][s + 1]):
                out["token_seq"].append(s)
                if out["status"][s]:
                    out["positions"].append(-1)
                    out["slots"].append(-1)
                else:
                    pos = int(past[s]) + i - out["query_start"][s]
                    out["positions"].append(pos)
                    out["slots"].append(int(self.tables[s, pos // B]) * B + pos % B)
        del self.free[free - last:]
        for k in ("positions", "token_seq", "slots"):
            out[k] += [-1] * (max_tokens - len(out[k]))
        return out


def norm_rope(x, w, eps, cos_sin, pos, interleaved):
    """64-bit norm and rotation of x [T][H][D]; also the sum of the absolute terms of each
    element, which bounds what roundings of 32 bits can do to it."""
    x = x.double()
    if w is not None:
        x = x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt() * w.double()
    size = x.abs()
    if cos_sin is None:
        return x, size
    r = cos_sin.shape[1]
    c, s = (t[:, None, :] for t in cos_sin[pos].double().split(r // 2, 1))
    out, size = x.clone(), size.clone()
    i = torch.arange(0, r, 2) if interleaved else torch.arange(r // 2)
    j = i + (1 if interleaved else r // 2)
    a, b = x[..., i], x[..., j]
    out[..., i], out[..., j] = a * c - b * s, b * c + a * s
    size[..., i] = (a * c).abs() + (b * s).abs()
    size[..., j] = (b * c).abs() + (a * s).abs()
    return out, size


def chunk_attention(q, k_pool, v_pool, query_start, tables, ctx, scale):
    """64-bit attention of every query row; also, for each output, the weighted mean of |V|
    (its error scale), the largest error 32-bit scores can have, and the context length."""
    T, Hq, D = q.shape
    N, Hkv, B, _ = k_pool.shape
    G = Hq // Hkv
    out = torch.zeros(T, Hq, D, dtype=torch.float64)
    mean_abs, delta = torch.zeros_like(out), torch.zeros(T, Hq, 1, dtype=torch.float64)
    length = torch.zeros(T, 1, 1, dtype=torch.float64)
    for s in range(len(ctx)):
        a, b, n = int(query_start[s]), int(query_start[s + 1]), int(ctx[s])
        if b <= a or n <= 0:
            continue
        ids = tables[s, :blocks(n, B)].long()
        for h in range(Hkv):
            k = k_pool[ids, h].reshape(-1, D)[:n].double()
            v = v_pool[ids, h].reshape(-1, D)[:n].double()
            x = q[a:b, h * G:(h + 1) * G].double()
            z = torch.einsum("tgd,nd->tgn", x, k) * scale
            seen = n - (b - a) + 1 + torch.arange(b - a)
            hidden = torch.arange(n)[None, :] >= seen[:, None]
            z = z.masked_fill(hidden[:, None, :], float("-inf"))
            real = (seen > 0)[:, None, None]
            p = torch.where(real, torch.softmax(torch.where(real, z, torch.zeros_like(z)), -1), 0.0)
            out[a:b, h * G:(h + 1) * G] = p @ v
            mean_abs[a:b, h * G:(h + 1) * G] = p @ v.abs()
            terms = torch.einsum("tgd,nd->tgn", x.abs(), k.abs()).amax(-1, keepdim=True) * abs(scale)
            delta[a:b, h * G:(h + 1) * G] = terms
        length[a:b] = n
    return out, mean_abs, delta, length


def chunk_tolerance(ref, mean_abs, delta, length, pool_dtype, out_dtype):
    """Largest |error| of a chunk output, from the roundings it goes through.

    u: half a step of the pool's type.  With weights p_i and sum l, out = sum p_i v_i / l:
    rounding each p_i to the pool's type changes out by at most u * A, A = sum p_i |v_i| / l
    (u^2 * A when the rounded remainder is added).  Scores: D-term products summed in 32
    bits, at most 128 * 2^-23 * terms off (the tensor cores may truncate: one whole step per
    addition), plus one rounding of a scaled score (|z| <= terms) in base 2; twice that,
    relative, on the weights and again on l.  Sums over `length` tokens in 32 bits: length *
    2^-23 relative to A, for O and for l.  2^-20 for the exponentials and divisions.  fp16
    weights below 2^-14 are subnormal: off by 2^-25 each, against l >= 1.  Last, half a step
    of the output's type."""
    u = torch.finfo(pool_dtype).eps / 2
    u_out = torch.finfo(out_dtype).eps / 2
    p_err = u if out_dtype == pool_dtype else u * u
    d = delta * (128 * 2.0 ** -23 + 2.0 ** -22)
    tol = mean_abs * (p_err + 2 * torch.expm1(d) + 2 * length * 2.0 ** -23 + 2.0 ** -20)
    if pool_dtype == torch.float16:
        tol = tol + length * 2.0 ** -25 * 8  # |v| < 8 in these tests
    return (tol + u_out * (ref.abs() + tol)) * (1 + 1e-6) + 1e-30
