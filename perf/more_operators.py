"""A paged cache held in 8 bits, operator by operator.

The cache's pages hold e4m3 values, and each page (a block of tokens of one key / value head) has a
32-bit scale for its keys and one for its values: a cached number is its 8-bit value times its
page's scale.  A request's tokens go through

  append  per-head norms of the queries and keys, their rotation by position, and the keys and
          values into their pages, whose scales grow where the new values need it
  decode  attention of one token, or the last few, of every request over its cached tokens
  chunk   causal attention of ragged prompts, or parts of them, over their cached tokens

Each operator has its plain form here, in torch operations on 32-bit values, and the call a user
makes of the library instead.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPE = {"f16": torch.float16, "bf16": torch.bfloat16}
CODE = torch.float8_e4m3fn
LARGEST = 448.0     # of the 8-bit type
LEAST_POWER = -100  # the least scale is 2 to this


# ---------------------------------------------------------------------------- cases

def listed():
    return [
        # one request's next token: the smallest call of a decoding engine
        dict(name="append_one", op="append", seqs=1, past=700, new=1, decode=1.0, heads=32, kv_heads=8, dim=128,
             block=16, dtype="bf16", norm=True, rotary=128, interleaved=False, pad=0, layout=11),
        # a decoding batch without shared heads or norms, pairs rotated side by side, room for a few more tokens
        dict(name="append_decode", op="append", seqs=128, past=500, new=1, decode=1.0, heads=40, kv_heads=40, dim=128,
             block=16, dtype="f16", norm=False, rotary=128, interleaved=True, pad=5, layout=12),
        # narrow heads, half of each rotated, prompts of all lengths that begin and end inside blocks
        dict(name="append_ragged", op="append", seqs=24, past=300, new=511, decode=0.2, heads=16, kv_heads=4, dim=64,
             block=32, dtype="f16", norm=True, rotary=32, interleaved=False, pad=3, layout=13),
        # the largest step: two prompts of 8192 tokens
        dict(name="append_prompts", op="append", seqs=2, past=0, new=8192, decode=0.0, heads=32, kv_heads=8, dim=128,
             block=16, dtype="bf16", norm=True, rotary=128, interleaved=False, pad=0, layout=0),
        # a handful of requests: latency
        dict(name="decode_few", op="decode", seqs=4, past=700, queries=1, heads=32, kv_heads=8, dim=128, block=16,
             dtype="bf16", layout=14),
        # narrow heads and four drafted tokens a request
        dict(name="decode_drafts", op="decode", seqs=64, past=400, queries=4, heads=16, kv_heads=4, dim=64, block=32,
             dtype="f16", layout=15),
        # a serving batch without shared heads
        dict(name="decode_batch", op="decode", seqs=128, past=600, queries=1, heads=40, kv_heads=40, dim=128, block=16,
             dtype="f16", layout=16),
        # very long contexts
        dict(name="decode_long", op="decode", seqs=8, past=80000, queries=1, heads=32, kv_heads=8, dim=128, block=16,
             dtype="bf16", layout=17),
        # narrow heads, prompts of all lengths beside decoding requests
        dict(name="chunk_ragged", op="chunk", seqs=24, past=300, new=512, decode=0.2, heads=16, kv_heads=4, dim=64,
             block=32, dtype="f16", layout=18),
        # one prompt of 8192 tokens from its first token
        dict(name="chunk_prompt", op="chunk", seqs=1, past=0, new=8192, decode=0.0, heads=32, kv_heads=8, dim=128,
             block=16, dtype="bf16", layout=0),
        # the next part of a very long prompt: few queries, a context of about 128k tokens
        dict(name="chunk_long", op="chunk", seqs=1, past=130000, new=500, decode=0.0, heads=32, kv_heads=8, dim=128,
             block=16, dtype="bf16", layout=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "chunk"])
    heads, kv_heads = rng.choice([(32, 8), (40, 40), (16, 4), (8, 1), (32, 32), (12, 6), (28, 4)])
    dim = rng.choice([64, 128, 128])
    case = dict(op=op, heads=heads, kv_heads=kv_heads, dim=dim, block=rng.choice([16, 32]),
                dtype=rng.choice(["bf16", "f16"]), layout=rng.randrange(1, 1 << 20))
    if op == "append":
        shape = rng.choice(["decode", "ragged", "prompts"])
        if shape == "decode":
            case.update(seqs=_log(rng, 1, 256), past=_log(rng, 16, 600), new=1, decode=1.0)
        elif shape == "ragged":
            case.update(seqs=rng.randint(2, 24), past=_log(rng, 8, 500), new=_log(rng, 2, 500),
                        decode=rng.choice([0.0, 0.3, 0.7]))
        else:
            case.update(seqs=1, past=rng.choice([0, 0, 333]), decode=0.0,
                        new=_log(rng, 500, 16384 * 48 // (heads + 2 * kv_heads)))
        case.update(norm=rng.random() < 0.6, rotary=rng.choice([dim, dim, dim // 2]), interleaved=rng.random() < 0.4,
                    pad=rng.choice([0, 0, 1, 7]))
    elif op == "decode":
        if rng.random() < 0.6:
            case.update(seqs=_log(rng, 1, 96), past=_log(rng, 1, 1200), queries=rng.choice([1, 1, 1, 2, 4, 7]))
        else:
            case.update(seqs=rng.randint(1, 3), past=_log(rng, 4000, 480000 // max(8, kv_heads)),
                        queries=rng.choice([1, 1, 3]))
    else:
        shape = rng.choice(["few", "ragged", "prompt", "long"])
        if shape == "few":
            case.update(seqs=rng.randint(1, 16), past=_log(rng, 16, 4000), new=rng.randint(1, 16), decode=0.5)
        elif shape == "ragged":
            case.update(seqs=rng.randint(8, 32), past=_log(rng, 64, 1200), new=_log(rng, 16, 400),
                        decode=rng.choice([0.2, 0.5]))
        elif shape == "prompt":
            case.update(seqs=1, past=rng.choice([0, 0, 333]), new=_log(rng, 500, 5000), decode=0.0)
        else:
            case.update(seqs=1, past=_log(rng, 8000, 40000), new=_log(rng, 1, 300), decode=0.0)
    return case


def _lengths(case):
    """(past, new) tokens of each request: part of the case, so that what a pass costs is too.
    layout 0: exactly the case's lengths; otherwise drawn around them, with the case's share
    of decoding requests (one new token)."""
    n, past = case["seqs"], case["past"]
    new = case.get("new") or case["queries"]
    if case["layout"] == 0:
        return [past] * n, [new] * n
    rng = random.Random(case["layout"])
    pasts, news = [], []
    for _ in range(n):
        pasts.append(min(4 * past, int(past * rng.lognormvariate(-0.3, 0.8))))
        if case["op"] == "decode":
            news.append(new)
        else:
            news.append(1 if rng.random() < case["decode"] else rng.randint(1, new))
    return pasts, news


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _blocks(n, block):
    return -(-n // block)


def _tables(lens, block, ids):
    """Block table rows (-1 past each request's blocks), the ids handed out in order."""
    width = max(1, max(_blocks(n, block) for n in lens))
    need = torch.tensor([_blocks(n, block) for n in lens], device=DEV)
    first = torch.cumsum(need, 0) - need
    j = torch.arange(width, device=DEV)
    at = first[:, None] + j[None, :]
    return torch.where(j[None, :] < need[:, None], ids[at.clamp(max=ids.numel() - 1)], -1).to(torch.int32)


def _power(p):
    """2 to whole numbers, as 32-bit values."""
    return ((p.to(torch.int32) + 127) << 23).view(torch.float32)


def _scale_for(top):
    """The least power of two whose 448 times reach `top`, but no less than the least scale."""
    m, e = torch.frexp(top)
    p = torch.where(m <= LARGEST / 512, e - 9, e - 8)
    return _power(torch.where(top > 0, p, LEAST_POWER).clamp(min=LEAST_POWER))


def _pool(N, Hkv, B, D, g):
    """A pool in use: every page filled, pages and heads of different size."""
    codes = torch.empty(N, Hkv, B, D, dtype=CODE, device=DEV)
    scale = torch.empty(N, Hkv, dtype=torch.float32, device=DEV)
    size = torch.exp(0.3 * torch.randn(1, Hkv, 1, 1, generator=g, device=DEV))
    for lo in range(0, N, 8192):
        x = torch.randn(min(8192, N - lo), Hkv, B, D, generator=g, device=DEV) * size
        s = _scale_for(x.abs().amax((2, 3)))
        codes[lo:lo + 8192] = (x / s[:, :, None, None]).to(CODE)
        scale[lo:lo + 8192] = s
    return codes, scale


def prepare(case, seed):
    S, Hq, Hkv, D, B = (case[k] for k in ("seqs", "heads", "kv_heads", "dim", "block"))
    g, dt = _gen(seed), DTYPE[case["dtype"]]
    pasts, news = _lengths(case)
    lens = [p + n for p, n in zip(pasts, news)]
    used = sum(_blocks(n, B) for n in lens)
    N = used + used // 10 + 1
    tables = _tables(lens, B, torch.randperm(N, generator=g, device=DEV).to(torch.int32))
    (k_pool, k_scale), (v_pool, v_scale) = _pool(N, Hkv, B, D, g), _pool(N, Hkv, B, D, g)
    cache = dict(k_pool=k_pool, v_pool=v_pool, k_scale=k_scale, v_scale=v_scale)
    starts = [0]
    for n in news:
        starts.append(starts[-1] + n)
    T = starts[-1]
    if case["op"] == "append":
        rows, start, past = T + case["pad"], _ints(starts), torch.tensor(pasts, device=DEV)
        t = torch.arange(T, device=DEV)
        seq = torch.searchsorted(start[1:].contiguous(), t.to(torch.int32), right=True)
        at = past[seq] + t - start[seq]
        # rows of a captured step that hold no token have neither position nor slot
        positions = torch.full((rows,), -1, dtype=torch.int32, device=DEV)
        slots = torch.full((rows,), -1, dtype=torch.int64, device=DEV)
        positions[:T] = at
        slots[:T] = tables[seq, at // B].long() * B + at % B
        # the output of the layer's query, key and value projection: one packed row a token
        packed = torch.randn(rows, (Hq + 2 * Hkv) * D, generator=g, device=DEV).to(dt)
        q, k, v = (x.view(rows, -1, D) for x in packed.split([Hq * D, Hkv * D, Hkv * D], 1))
        rot, far = case["rotary"], max(lens)
        inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
        angle = torch.arange(far, dtype=torch.float64, device=DEV)[:, None] * inv[None, :]
        cos_sin = torch.cat([torch.cos(angle), torch.sin(angle)], 1).to(torch.float32)
        weights = [None, None]
        if case["norm"]:
            weights = [(1 + 0.2 * torch.randn(D, generator=g, device=DEV)).to(dt) for _ in range(2)]
        return dict(op="append", **cache, q=q, k=k, v=v, positions=positions, slots=slots, cos_sin=cos_sin,
                    wq=weights[0], wk=weights[1], eps=1e-6, interleaved=case["interleaved"],
                    q_out=torch.zeros(rows, Hq, D, dtype=dt, device=DEV))
    shape = (S, case["queries"], Hq, D) if case["op"] == "decode" else (T, Hq, D)
    return dict(op=case["op"], **cache, q=torch.randn(*shape, generator=g, device=DEV).to(dt), tables=tables,
                context=_ints(lens), query_start=_ints(starts), scale=D ** -0.5, longest=max(lens), most_new=max(news),
                out=torch.zeros(*shape, dtype=dt, device=DEV))


# ---------------------------------------------------------------------------- one pass

def run(s):
    if own:
        return {"append": _own_append, "decode": _own_decode, "chunk": _own_chunk}[s["op"]](s)
    return {"append": _plain_append, "decode": _plain_decode, "chunk": _plain_chunk}[s["op"]](s)


def _append_outputs(s):
    return {"q": s["q_out"], "k_pool": s["k_pool"], "v_pool": s["v_pool"], "k_scale": s["k_scale"],
            "v_scale": s["v_scale"]}


def _own_append(s):
    from paged_kv_cache_293_gb300 import pagedkv as P
    P.pkv_qk_norm_rope_write_q8(s["q"], s["k"], s["v"], s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"],
                                s["positions"], s["slots"], s["q_out"], q_weight=s["wq"], k_weight=s["wk"],
                                eps=s["eps"], cos_sin=s["cos_sin"], interleaved=s["interleaved"])
    return _append_outputs(s)


def _own_decode(s):
    from paged_kv_cache_293_gb300 import pagedkv as P
    ws = s.get("workspace")
    if ws is None:
        S, NQ, Hq, _ = s["q"].shape
        ws = s["workspace"] = P.workspace_tensor(
            P.pkv_decode_q8_workspace_bytes(s["k_pool"], S, NQ, Hq, s["longest"]), DEV)
    P.pkv_paged_attention_decode_q8(s["q"], s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], s["tables"],
                                    s["context"], s["scale"], s["out"], s["longest"], workspace=ws)
    return {"out": s["out"]}


def _own_chunk(s):
    from paged_kv_cache_293_gb300 import pagedkv as P
    ws = s.get("workspace")
    if ws is None:
        T, Hq, _ = s["q"].shape
        ws = s["workspace"] = P.workspace_tensor(
            P.pkv_chunk_q8_workspace_bytes(s["k_pool"], T, s["context"].numel(), Hq, s["longest"]), DEV)
    P.pkv_paged_attention_chunk_q8(s["q"], s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], s["query_start"],
                                   s["tables"], s["context"], s["scale"], s["out"], s["longest"], ws)
    return {"out": s["out"]}


def _plain_norm_rope(x, weight, eps, cos, sin, interleaved):
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * weight.float()
    half = cos.shape[-1]
    turned, kept = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = turned[..., :half], turned[..., half:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, kept], -1)


def _plain_into_pages(x, pool, scale, blocks, page, row):
    """The tokens' rows x into `page` of the touched `blocks`, at `row`: a block that gets its first row
    takes the scale that the new values need, another one the larger of that and its own, to which
    the rows it holds are rounded again."""
    U, Hkv = blocks.numel(), x.shape[1]
    top = torch.zeros(U, Hkv, device=DEV).scatter_reduce_(0, page[:, None].expand(-1, Hkv), x.abs().amax(-1), "amax")
    first = torch.full((U,), pool.shape[2], device=DEV).scatter_reduce_(0, page, row, "amin")
    old, need = scale[blocks], _scale_for(top)
    s = torch.where((first > 0)[:, None], torch.maximum(old, need), need)
    grown = (first > 0)[:, None] & (s > old)
    pages = pool[blocks].float()
    pages = torch.where(grown[:, :, None, None], pages * (old / s)[:, :, None, None], pages)
    pages = pages.to(CODE).float()
    pages[page, :, row] = (x / s[page][:, :, None]).to(CODE).float()
    pool[blocks] = pages.to(CODE)
    scale[blocks] = s


def _plain_append(s):
    q, k, pos, slots = s["q"], s["k"], s["positions"].long(), s["slots"]
    rows = s["cos_sin"][pos.clamp(min=0)]
    half = rows.shape[1] // 2
    cos, sin = rows[:, None, :half], rows[:, None, half:]
    turned = _plain_norm_rope(q, s["wq"], s["eps"], cos, sin, s["interleaved"]).to(q.dtype)
    s["q_out"].copy_(torch.where((pos >= 0)[:, None, None], turned, s["q_out"]))
    turned = _plain_norm_rope(k, s["wk"], s["eps"], cos, sin, s["interleaved"])
    real = (pos >= 0) & (slots >= 0)
    B = s["k_pool"].shape[2]
    blocks, page = torch.unique_consecutive(slots[real] // B, return_inverse=True)
    row = slots[real] % B
    _plain_into_pages(turned[real], s["k_pool"], s["k_scale"], blocks, page, row)
    _plain_into_pages(s["v"][real].float(), s["v_pool"], s["v_scale"], blocks, page, row)
    return _append_outputs(s)


def _plain_attention(s, qs, new):
    """qs [S][J][Hq][D]: query j of the J rows of a request sees its context but the last
    new - 1 - j positions.  All requests at once, padded to the longest context."""
    S, J, Hq, D = qs.shape
    Hkv = s["k_pool"].shape[1]
    G, ctx = Hq // Hkv, s["context"].long()
    blocks = s["tables"].long().clamp(min=0)

    def cached(pool, scale):
        x = pool[blocks].float() * scale[blocks][..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(S, Hkv, -1, D)

    k = cached(s["k_pool"], s["k_scale"])
    qs = qs.view(S, J, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(S, Hkv, -1, D).float()
    scores = (qs @ k.transpose(-1, -2)).view(S, Hkv, G, J, -1) * s["scale"]
    seen = (ctx - new)[:, None] + 1 + torch.arange(J, device=DEV)[None, :]
    hidden = torch.arange(k.shape[2], device=DEV)[None, None, :] >= seen[:, :, None]
    del k
    scores = scores.masked_fill_(hidden[:, None, None], float("-inf"))
    top = scores.amax(-1, keepdim=True)
    p = scores.sub_(torch.where(top == float("-inf"), 0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    v = cached(s["v_pool"], s["v_scale"])
    out = (p.view(S, Hkv, -1, v.shape[2]) @ v).view(S, Hkv, G, J, D)
    out = out / torch.where(total > 0, total, 1)
    return out.permute(0, 3, 1, 2, 4).reshape(S, J, Hq, D)


def _plain_decode(s):
    out = _plain_attention(s, s["q"], torch.full_like(s["context"], s["q"].shape[1]).long())
    s["out"].copy_(out.to(s["q"].dtype))
    return {"out": s["out"]}


def _plain_chunk(s):
    q, start = s["q"], s["query_start"].long()
    T, S = q.shape[0], s["context"].numel()
    j = torch.arange(s["most_new"], device=DEV)
    rows = (start[:-1, None] + j[None, :]).clamp(max=T - 1)
    out = _plain_attention(s, q[rows], start[1:] - start[:-1])
    t = torch.arange(T, device=DEV)
    seq = torch.searchsorted(start[1:].contiguous(), t, right=True).clamp(max=S - 1)
    s["out"].copy_(out[seq, t - start[seq]].to(q.dtype))
    return {"out": s["out"]}


# ---------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    Hq, Hkv, D, B = case["heads"], case["kv_heads"], case["dim"], case["block"]
    pasts, news = _lengths(case)
    if case["op"] == "append":
        T = sum(news)
        pages = sum(_blocks(p + n, B) - p // B for p, n in zip(pasts, news))
        # rows in, q out in 16 bits, k and v out in 8, each token's cosines and sines, position and
        # slot, and the scales of the pages that get tokens, in and out
        return {"bytes": T * ((2 * Hq + 2 * Hkv) * D * 2 + 2 * Hkv * D + 4 * case["rotary"] + 12) + pages * Hkv * 16,
                "flops": T * (Hq + Hkv) * D * (8 if case["norm"] else 4)}
    cached = sum(pasts) + sum(news)
    pages = sum(_blocks(p + n, B) for p, n in zip(pasts, news))
    pairs = sum(p * n + n * (n + 1) // 2 for p, n in zip(pasts, news))
    return {"bytes": 2 * sum(news) * Hq * D * 2 + 2 * cached * Hkv * D + pages * (8 * Hkv + 4),
            "flops": 4 * pairs * Hq * D}


# ---------------------------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    q, out = s["q"].flatten(0, -3), torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    flat = out.view(q.shape)
    starts, ctx = s["query_start"].tolist(), s["context"].tolist()
    _, Hkv, B, D = s["k_pool"].shape
    G = q.shape[1] // Hkv
    for i, n in enumerate(ctx):
        a, b = starts[i], starts[i + 1]
        ids = s["tables"][i, :_blocks(n, B)].long()
        for h in range(Hkv):
            k, v = ((s[x + "_pool"][ids, h].double() * s[x + "_scale"][ids, h].double()[:, None, None]).view(-1, D)[:n]
                    for x in "kv")
            for head in range(h * G, (h + 1) * G):
                for lo in range(a, b, 2048):
                    hi = min(b, lo + 2048)
                    z = torch.einsum("td,nd->tn", q[lo:hi, head].double(), k) * s["scale"]
                    last = n - b + torch.arange(lo, hi, device=DEV)
                    z[torch.arange(n, device=DEV)[None, :] > last[:, None]] = float("-inf")
                    flat[lo:hi, head] = torch.softmax(z, -1) @ v
    return {"out": out}


def _exact_code(x):
    """x at the nearest 8-bit value (three bits behind the first, steps of at least 2^-9), even at ties."""
    _, e = torch.frexp(x)
    step = torch.pow(2.0, (e - 4).clamp(min=-9).double())
    return torch.round(x / step) * step


def _exact_append(s):
    real = s["positions"] >= 0
    pos, slots = s["positions"][real].long(), s["slots"][real]
    table = s["cos_sin"][pos].double()
    half = table.shape[1] // 2
    turn = torch.complex(table[:, :half], table[:, half:])[:, None, :]
    done = []
    for x, w in ((s["q"][real], s["wq"]), (s["k"][real], s["wk"])):
        x = x.double()
        if w is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + s["eps"]).sqrt() * w.double()
        x = x.clone()
        if s["interleaved"]:
            a, b = x[..., 0:2 * half:2].clone(), x[..., 1:2 * half:2].clone()
        else:
            a, b = x[..., :half].clone(), x[..., half:2 * half].clone()
        z = torch.complex(a, b) * turn
        if s["interleaved"]:
            x[..., 0:2 * half:2], x[..., 1:2 * half:2] = z.real, z.imag
        else:
            x[..., :half], x[..., half:2 * half] = z.real, z.imag
        done.append(x)
    q = s["q_out"].double()
    q[real] = done[0]
    outs = {"q": q}
    N, Hkv, B, D = s["k_pool"].shape
    block, row = slots // B, slots % B
    got = torch.zeros(N, dtype=torch.bool, device=DEV)
    got[block] = True
    begins = torch.zeros(N, dtype=torch.bool, device=DEV)
    begins[block[row == 0]] = True
    for name, new in (("k", done[1]), ("v", s["v"][real].double())):
        codes, scale = s[name + "_pool"].double(), s[name + "_scale"].double()
        top = torch.zeros(N, Hkv, dtype=torch.float64, device=DEV)
        top.scatter_reduce_(0, block[:, None].expand(-1, Hkv), new.abs().amax(-1), "amax")
        power = torch.ceil(torch.log2(top.clamp(min=1e-300) / LARGEST)).clamp(min=LEAST_POWER)
        need = torch.pow(2.0, power)
        s2 = torch.where(got[:, None], torch.where(begins[:, None], need, torch.maximum(scale, need)), scale)
        more = got[:, None] & ~begins[:, None] & (s2 > scale)
        codes = torch.where(more[:, :, None, None], _exact_code(codes * (scale / s2)[:, :, None, None]), codes)
        codes[block, :, row] = _exact_code(new / s2[block][:, :, None])
        outs[name + "_pool"], outs[name + "_scale"] = codes, s2
    return outs
