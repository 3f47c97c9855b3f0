"""One ragged step of a paged-cache engine, operator by operator.

A step serves requests with any number of new tokens each (one for a decoding request,
up to thousands for a prompt or a part of one), packed behind one another:

  batch   from the request lengths alone: block tables, query starts, positions and slots
  write   per-head norms of the queries and keys, their rotation by position, and the keys
          and values into their cache slots
  attend  causal attention of every new token over its request's cached tokens

Each operator has its plain form here, in torch operations on 32-bit values (whole numbers
where the operator has whole numbers), and the call a user makes of the library instead.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPE = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------- cases

def listed():
    return [
        # four short requests at the very start of serving: latency only
        dict(name="batch_tiny", op="batch", seqs=4, past=100, new=60, decode=0.0, block=16, layout=1),
        # a decoding engine's step: one new token for each of 128 requests
        dict(name="batch_decode", op="batch", seqs=128, past=1024, new=1, decode=1.0, block=16, layout=2),
        # thousands of requests, most decoding and the rest with long prompts
        dict(name="batch_large", op="batch", seqs=4096, past=2048, new=512, decode=0.75, block=32, layout=3),
        # one token of one request (the smallest call a decoding engine makes)
        dict(name="write_one", op="write", tokens=1, heads=32, kv_heads=8, dim=128, block=16, dtype="bf16",
             norm=True, rotary=128, interleaved=False, max_pos=131072, pad=0, layout=4),
        # a decoding batch without shared heads or norms, pairs rotated side by side
        dict(name="write_decode", op="write", tokens=128, heads=40, kv_heads=40, dim=128, block=16, dtype="f16",
             norm=False, rotary=128, interleaved=True, max_pos=4096, pad=5, layout=5),
        # 32-bit values, narrow heads, half of each head rotated, an odd number of tokens
        dict(name="write_f32", op="write", tokens=777, heads=4, kv_heads=4, dim=64, block=16, dtype="f32",
             norm=True, rotary=32, interleaved=False, max_pos=2048, pad=3, layout=6),
        # the largest step: prompts of 16384 tokens in all
        dict(name="write_prompts", op="write", tokens=16384, heads=32, kv_heads=8, dim=128, block=16, dtype="bf16",
             norm=True, rotary=128, interleaved=False, max_pos=131072, pad=0, layout=7),
        # a handful of requests with a few new tokens each: latency
        dict(name="attend_few", op="attend", seqs=6, past=700, new=5, decode=0.5, heads=32, kv_heads=8, dim=128,
             block=16, dtype="bf16", layout=8),
        # narrow heads, prompts of all lengths
        dict(name="attend_narrow", op="attend", seqs=24, past=300, new=512, decode=0.2, heads=16, kv_heads=4, dim=64,
             block=32, dtype="f16", layout=9),
        # a mixed step of an engine without shared heads: decoding requests beside parts of prompts
        dict(name="attend_mixed", op="attend", seqs=48, past=1500, new=400, decode=0.7, heads=40, kv_heads=40, dim=128,
             block=16, dtype="f16", layout=10),
        # one prompt of 8192 tokens from its first token
        dict(name="attend_prompt", op="attend", seqs=1, past=0, new=8192, decode=0.0, heads=32, kv_heads=8, dim=128,
             block=16, dtype="bf16", layout=0),
        # the next part of a very long prompt: few queries, a context of about 128k tokens
        dict(name="attend_long", op="attend", seqs=1, past=130000, new=500, decode=0.0, heads=32, kv_heads=8, dim=128,
             block=16, dtype="bf16", layout=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["batch", "write", "attend", "attend"])
    layout = rng.randrange(1, 1 << 20)
    if op == "batch":
        seqs = _log(rng, 1, 4096)
        return dict(op=op, seqs=seqs, past=_log(rng, 16, 2048), new=_log(rng, 1, 512),
                    decode=rng.choice([0.0, 0.5, 0.75, 1.0]), block=rng.choice([16, 32]), layout=layout)
    heads, kv_heads = rng.choice([(32, 8), (40, 40), (16, 4), (8, 1), (32, 32), (12, 6), (28, 4)])
    dim = rng.choice([64, 128, 128])
    if op == "write":
        tokens = _log(rng, 1, 16384 * 48 // (heads + 2 * kv_heads))
        return dict(op=op, tokens=tokens, heads=heads, kv_heads=kv_heads, dim=dim, block=rng.choice([16, 32]),
                    dtype=rng.choice(["bf16", "f16", "bf16", "f32"]) if tokens < 4000 else rng.choice(["bf16", "f16"]),
                    norm=rng.random() < 0.6, rotary=rng.choice([dim, dim, dim // 2]), interleaved=rng.random() < 0.4,
                    max_pos=_log(rng, 512, 131072), pad=rng.choice([0, 0, 1, 7]), layout=layout)
    shape = rng.choice(["few", "ragged", "prompt", "long"])
    if shape == "few":
        seqs, past, new, decode = rng.randint(1, 16), _log(rng, 16, 4000), rng.randint(1, 16), 0.5
    elif shape == "ragged":
        seqs, past, new, decode = rng.randint(8, 48), _log(rng, 64, 1200), _log(rng, 16, 400), rng.choice([0.2, 0.5, 0.7])
    elif shape == "prompt":
        seqs, past, new, decode = 1, rng.choice([0, 0, 333]), _log(rng, 500, 5000), 0.0
    else:
        seqs, past, new, decode = 1, _log(rng, 8000, 100000), _log(rng, 1, 350), 0.0
    return dict(op=op, seqs=seqs, past=past, new=new, decode=decode, heads=heads, kv_heads=kv_heads, dim=dim,
                block=rng.choice([16, 32]), dtype=rng.choice(["bf16", "f16"]), layout=layout)


def _lengths(case):
    """(past, new) tokens of each request: part of the case, so that what a pass costs is too.
    layout 0: exactly the case's lengths; otherwise drawn around them, with the case's share
    of decoding requests (one new token)."""
    n, past, new = case["seqs"], case["past"], case["new"]
    if case["layout"] == 0:
        return [past] * n, [new] * n
    rng = random.Random(case["layout"])
    pasts, news = [], []
    for _ in range(n):
        p = min(4 * past, int(past * rng.lognormvariate(-0.3, 0.8)))
        m = 1 if rng.random() < case["decode"] else rng.randint(1, new)
        pasts.append(p)
        news.append(m)
    return pasts, news


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=DEV)


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


def prepare(case, seed):
    return {"batch": _prepare_batch, "write": _prepare_write, "attend": _prepare_attend}[case["op"]](case, seed)


def _prepare_batch(case, seed):
    B = case["block"]
    pasts, news = _lengths(case)
    S, g = case["seqs"], _gen(seed)
    held = sum(_blocks(p, B) for p in pasts)
    grown = sum(_blocks(p + n, B) for p, n in zip(pasts, news))
    N = grown + max(4, grown // 10)
    ids = torch.randperm(N, generator=g, device=DEV).to(torch.int32)
    width = max(_blocks(p + n, B) for p, n in zip(pasts, news)) + 1
    tables = torch.full((S, width), -1, dtype=torch.int32, device=DEV)
    old = _tables(pasts, B, ids)
    tables[:, :old.shape[1]] = old[:, :width]
    free_ids = torch.full((N,), -1, dtype=torch.int32, device=DEV)
    free_ids[:N - held] = ids[held:]
    refcount = torch.zeros(N, dtype=torch.int32, device=DEV)
    refcount[ids[:held].long()] = 1
    cap = sum(news) + 8  # a step captured into a graph has room for a few tokens more
    i32 = dict(dtype=torch.int32, device=DEV)
    return dict(op="batch", B=B, cap=cap, tables=tables, past=_ints(pasts), new=_ints(news), free_ids=free_ids,
                free_count=_ints([N - held]), refcount=refcount, free_left=torch.zeros(1, **i32),
                query_start=torch.zeros(S + 1, **i32), context=torch.zeros(S, **i32), positions=torch.zeros(cap, **i32),
                token_seq=torch.zeros(cap, **i32), slots=torch.zeros(cap, dtype=torch.int64, device=DEV),
                status=torch.zeros(S, **i32))


def _prepare_write(case, seed):
    T, Hq, Hkv, D, B = (case[k] for k in ("tokens", "heads", "kv_heads", "dim", "block"))
    g, dt = _gen(seed), DTYPE[case["dtype"]]
    rows = T + case["pad"]
    # the output of the layer's query, key and value projection: one packed row a token
    packed = torch.randn(rows, (Hq + 2 * Hkv) * D, generator=g, device=DEV).to(dt)
    q = packed[:, :Hq * D].view(rows, Hq, D)
    k = packed[:, Hq * D:(Hq + Hkv) * D].view(rows, Hkv, D)
    v = packed[:, (Hq + Hkv) * D:].view(rows, Hkv, D)
    N = _blocks(T, B) + 2 + _blocks(T, B) // 10
    slots = torch.randperm(N * B, generator=g, device=DEV)[:rows].clone()
    slots[T:] = -1
    start = torch.randint(0, case["max_pos"], (1,), generator=g, device=DEV)
    positions = ((start + torch.arange(rows, device=DEV)) % case["max_pos"]).to(torch.int32)
    positions[T:] = -1  # rows of a captured step that hold no token
    rot = case["rotary"]
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    angle = torch.arange(case["max_pos"], dtype=torch.float64, device=DEV)[:, None] * inv[None, :]
    cos_sin = torch.cat([torch.cos(angle), torch.sin(angle)], 1).to(torch.float32)
    weights = [None, None]
    if case["norm"]:
        weights = [(1 + 0.2 * torch.randn(D, generator=g, device=DEV)).to(dt) for _ in range(2)]
    return dict(op="write", q=q, k=k, v=v, positions=positions, slots=slots, cos_sin=cos_sin, wq=weights[0],
                wk=weights[1], eps=1e-6, interleaved=case["interleaved"],
                k_pool=torch.zeros(N, Hkv, B, D, dtype=dt, device=DEV),
                v_pool=torch.zeros(N, Hkv, B, D, dtype=dt, device=DEV),
                q_out=torch.zeros(rows, Hq, D, dtype=dt, device=DEV))


def _prepare_attend(case, seed):
    S, Hq, Hkv, D, B = (case[k] for k in ("seqs", "heads", "kv_heads", "dim", "block"))
    g, dt = _gen(seed), DTYPE[case["dtype"]]
    pasts, news = _lengths(case)
    lens = [p + n for p, n in zip(pasts, news)]
    used = sum(_blocks(n, B) for n in lens)
    N = used + used // 10 + 1
    ids = torch.randperm(N, generator=g, device=DEV).to(torch.int32)
    starts = [0]
    for n in news:
        starts.append(starts[-1] + n)
    T = starts[-1]
    k_pool, v_pool = (torch.randn(N, Hkv, B, D, generator=g, device=DEV, dtype=torch.float32).to(dt) for _ in range(2))
    return dict(op="attend", q=torch.randn(T, Hq, D, generator=g, device=DEV).to(dt), k_pool=k_pool, v_pool=v_pool,
                tables=_tables(lens, B, ids), query_start=_ints(starts), context=_ints(lens), scale=D ** -0.5,
                longest=max(lens), most_new=max(news), out=torch.zeros(T, Hq, D, dtype=dt, device=DEV))


# ---------------------------------------------------------------------------- one pass

def run(s):
    if own:
        return {"batch": _own_batch, "write": _own_write, "attend": _own_attend}[s["op"]](s)
    return {"batch": _plain_batch, "write": _plain_write, "attend": _plain_attend}[s["op"]](s)


def _batch_outputs(s):
    return {k: s[k] for k in ("tables", "refcount", "free_left", "query_start", "context", "positions", "token_seq",
                              "slots", "status")}


def _own_batch(s):
    from paged_kv_cache_293_gb300 import pagedkv as P
    alloc = s.get("alloc")
    if alloc is None:
        alloc = s["alloc"] = P.BlockAllocator.of_tensors(s["free_ids"], s["free_count"], s["refcount"])
    P.pkv_build_batch(alloc, s["B"], s["tables"], s["past"], s["new"], s["query_start"], s["context"], s["positions"],
                      s["token_seq"], s["slots"], s["status"], free_count_out=s["free_left"])
    return _batch_outputs(s)


def _own_write(s):
    from paged_kv_cache_293_gb300 import pagedkv as P
    P.pkv_qk_norm_rope_write(s["q"], s["k"], s["v"], s["k_pool"], s["v_pool"], s["positions"], s["slots"], s["q_out"],
                             q_weight=s["wq"], k_weight=s["wk"], eps=s["eps"], cos_sin=s["cos_sin"],
                             interleaved=s["interleaved"])
    return {"q": s["q_out"], "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def _own_attend(s):
    from paged_kv_cache_293_gb300 import pagedkv as P
    ws = s.get("workspace")
    if ws is None:
        n = P.pkv_chunk_workspace_bytes(s["k_pool"], s["q"].shape[0], s["context"].numel(), s["q"].shape[1], s["longest"])
        ws = s["workspace"] = P.workspace_tensor(n, DEV)
    P.pkv_paged_attention_chunk(s["q"], s["k_pool"], s["v_pool"], s["query_start"], s["tables"], s["context"], s["scale"],
                                s["out"], s["longest"], ws)
    return {"out": s["out"]}


def _plain_batch(s):
    """Requests are served in order while the free blocks last; here all of them fit."""
    B, past, new, tables = s["B"], s["past"].long(), s["new"].long(), s["tables"]
    held, grown = (past + B - 1) // B, (past + new + B - 1) // B
    need = grown - held
    upto = torch.cumsum(need, 0)
    free = s["free_count"].long()
    served = (need == 0) | (upto <= free)
    need = torch.where(served, need, 0)
    first = upto - need
    j = torch.arange(tables.shape[1], device=DEV)[None, :]
    fresh = (j >= held[:, None]) & (j < (held + need)[:, None])
    rank = first[:, None] + j - held[:, None]
    ids = s["free_ids"][(free - 1 - rank).clamp(0, s["free_ids"].numel() - 1)]
    tables.copy_(torch.where(fresh, ids, tables))
    counts = torch.zeros(s["refcount"].numel() + 1, dtype=torch.int32, device=DEV)
    counts[torch.where(fresh, ids, s["refcount"].numel()).long().reshape(-1)] = 1
    s["refcount"].copy_(torch.where(counts[:-1] > 0, 1, s["refcount"]))
    s["free_left"].copy_(free - need.sum())
    starts = torch.cumsum(new, 0)
    s["query_start"][0] = 0
    s["query_start"][1:] = starts
    s["context"].copy_(torch.where(served, past + new, 0))
    s["status"].copy_(torch.where(served, 0, 1))
    t = torch.arange(s["cap"], device=DEV)
    seq = torch.searchsorted(starts, t, right=True)
    real = seq < past.numel()
    at = seq.clamp(max=past.numel() - 1)
    p = past[at] + t - (starts - new)[at]
    p = torch.where(real & served[at], p, -1)
    block = tables[at, (p.clamp(min=0) // B)].long()
    s["positions"].copy_(p)
    s["token_seq"].copy_(torch.where(real, seq, -1))
    s["slots"].copy_(torch.where(p >= 0, block * B + p % B, -1))
    return _batch_outputs(s)


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


def _plain_write(s):
    q, k, v, pos, slots = s["q"], s["k"], s["v"], s["positions"].long(), s["slots"]
    rows = s["cos_sin"][pos.clamp(min=0)]
    half = rows.shape[1] // 2
    cos, sin = rows[:, None, :half], rows[:, None, half:]
    real = (pos >= 0)[:, None, None]
    turned = _plain_norm_rope(q, s["wq"], s["eps"], cos, sin, s["interleaved"]).to(q.dtype)
    s["q_out"].copy_(torch.where(real, turned, s["q_out"]))
    N, Hkv, B, D = s["k_pool"].shape
    turned = _plain_norm_rope(k, s["wk"], s["eps"], cos, sin, s["interleaved"]).to(k.dtype)
    # rows without a token go to a spare row behind the pool's
    at = torch.where((pos >= 0) & (slots >= 0), slots, N * B)
    for pool, new in ((s["k_pool"], turned), (s["v_pool"], v)):
        flat = torch.cat([pool.transpose(1, 2).reshape(N * B, Hkv, D), pool.new_zeros(1, Hkv, D)])
        flat[at] = new
        pool.copy_(flat[:-1].view(N, B, Hkv, D).transpose(1, 2))
    return {"q": s["q_out"], "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def _plain_attend(s):
    """All requests at once, padded to the longest context and the most new tokens."""
    q, start, ctx = s["q"], s["query_start"].long(), s["context"].long()
    N, Hkv, B, D = s["k_pool"].shape
    T, Hq, _ = q.shape
    S, G = ctx.numel(), Hq // Hkv
    new = start[1:] - start[:-1]
    blocks = s["tables"].long().clamp(min=0)
    k = s["k_pool"][blocks].permute(0, 2, 1, 3, 4).reshape(S, Hkv, -1, D).float()
    v = s["v_pool"][blocks].permute(0, 2, 1, 3, 4).reshape(S, Hkv, -1, D).float()
    j = torch.arange(s["most_new"], device=DEV)
    rows = (start[:-1, None] + j[None, :]).clamp(max=T - 1)
    qs = q[rows].view(S, -1, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(S, Hkv, -1, D).float()
    scores = (qs @ k.transpose(-1, -2)).view(S, Hkv, G, j.numel(), -1) * s["scale"]
    seen = (ctx - new)[:, None] + 1 + j[None, :]
    hidden = torch.arange(k.shape[2], device=DEV)[None, None, :] >= seen[:, :, None]
    scores = scores.masked_fill_(hidden[:, None, None], float("-inf"))
    top = scores.amax(-1, keepdim=True)
    p = scores.sub_(torch.where(top == float("-inf"), 0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p.view(S, Hkv, -1, k.shape[2]) @ v).view(S, Hkv, G, j.numel(), D)
    out = out / torch.where(total > 0, total, 1)
    out = out.permute(0, 3, 1, 2, 4).reshape(S, j.numel(), Hq, D)
    t = torch.arange(T, device=DEV)
    seq = torch.searchsorted(start[1:].contiguous(), t, right=True).clamp(max=S - 1)
    s["out"].copy_(out[seq, t - start[seq]].to(q.dtype))
    return {"out": s["out"]}


# ---------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    e = 4 if case.get("dtype") == "f32" else 2
    if case["op"] == "batch":
        B = case["block"]
        pasts, news = _lengths(case)
        fresh = sum(_blocks(p + n, B) - _blocks(p, B) for p, n in zip(pasts, news))
        tokens, S = sum(news) + 8, case["seqs"]
        # lengths in; starts, contexts and statuses out; ids in, table entries and counts out;
        # a position, a request and a slot a token out
        return {"bytes": 8 * S + 12 * S + 12 * fresh + 16 * tokens, "flops": 0}
    Hq, Hkv, D = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "write":
        T = case["tokens"]
        # every row in and out, its rotation's cosines and sines, its position and slot
        return {"bytes": T * (2 * (Hq + 2 * Hkv) * D * e + 4 * case["rotary"] + 12),
                "flops": T * (Hq + Hkv) * D * (8 if case["norm"] else 4)}
    pasts, news = _lengths(case)
    tokens, cached = sum(news), sum(pasts) + sum(news)
    pairs = sum(p * n + n * (n + 1) // 2 for p, n in zip(pasts, news))
    return {"bytes": 2 * tokens * Hq * D * e + 2 * cached * Hkv * D * e, "flops": 4 * pairs * Hq * D}


# ---------------------------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    if case["op"] == "batch":
        return None  # whole numbers only
    s = prepare(case, seed)
    if case["op"] == "write":
        return _exact_write(s)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    starts, ctx = s["query_start"].tolist(), s["context"].tolist()
    N, Hkv, B, D = s["k_pool"].shape
    G = s["q"].shape[1] // Hkv
    for i, n in enumerate(ctx):
        a, b = starts[i], starts[i + 1]
        ids = s["tables"][i, :_blocks(n, B)].long()
        for h in range(Hkv):
            k = s["k_pool"][ids, h].reshape(-1, D)[:n].double()
            v = s["v_pool"][ids, h].reshape(-1, D)[:n].double()
            for g in range(h * G, (h + 1) * G):
                for lo in range(a, b, 2048):
                    hi = min(b, lo + 2048)
                    z = torch.einsum("td,nd->tn", s["q"][lo:hi, g].double(), k) * s["scale"]
                    last = n - b + torch.arange(lo, hi, device=DEV)
                    z[torch.arange(n, device=DEV)[None, :] > last[:, None]] = float("-inf")
                    out[lo:hi, g] = torch.softmax(z, -1) @ v
    return {"out": out}


def _exact_write(s):
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
    pools = []
    B = s["k_pool"].shape[2]
    for pool, new in ((s["k_pool"], done[1]), (s["v_pool"], s["v"][real].double())):
        pool = pool.double()
        pool[slots // B, :, slots % B] = new
        pools.append(pool)
    return {"q": q, "k_pool": pools[0], "v_pool": pools[1]}
