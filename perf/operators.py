"""Work of the packed and paged attention operators, for timing and for comparing outputs.

Five operators, as a serving or training program calls them:

    prompt   attn_fwd_packed: attention over whole prompts of different
             lengths packed one behind the other, grouped heads
    train    attn_fwd_packed, then attn_bwd_packed: a training step's
             attention with its gradients
    chunk    attn_chunk_paged: the new tokens of each request (one, or a
             chunk of a prompt) over a paged cache
    plan     attn_paged_plan: block tables and slot maps from request lengths
    write    attn_paged_write: new K and V rows into the pages, by slot

Where ``own`` is false, ``run`` computes them with elementary torch
operations in fp32; where it is true, it calls the library.
"""
import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a handful of short requests that arrive together: the call's own latency counts
        {"name": "prompt short", "op": "prompt", "b": 3, "shortest": 7, "longest": 150, "h": 16, "h_kv": 4,
         "d": 64, "dtype": "fp16", "causal": True, "fused": False, "lens": 1},
        # an ordinary prefill batch, q, k and v as slices of one projection
        {"name": "prompt batch", "op": "prompt", "b": 16, "shortest": 64, "longest": 1500, "h": 32, "h_kv": 8,
         "d": 128, "dtype": "bf16", "causal": True, "fused": True, "lens": 2},
        # long documents
        {"name": "prompt long", "op": "prompt", "b": 2, "shortest": 7777, "longest": 8192, "h": 32, "h_kv": 8,
         "d": 128, "dtype": "bf16", "causal": True, "fused": False, "lens": 3},
        # a training step of a small model: every head its own K/V, odd lengths
        {"name": "train short", "op": "train", "b": 5, "shortest": 33, "longest": 301, "h": 16, "h_kv": 16,
         "d": 64, "dtype": "fp16", "causal": True, "fused": False, "lens": 4},
        # a training step over documents packed into one row
        {"name": "train packed", "op": "train", "b": 6, "shortest": 200, "longest": 4096, "h": 32, "h_kv": 8,
         "d": 128, "dtype": "bf16", "causal": True, "fused": True, "lens": 5},
        # one user, one new token: latency
        {"name": "decode one", "op": "chunk", "b": 1, "chunks": 0, "chunk": 1, "shortest": 900, "longest": 900,
         "page": 16, "h": 32, "h_kv": 8, "d": 128, "dtype": "bf16", "lens": 6},
        # a full decode batch, one token each, caches of very different lengths
        {"name": "decode batch", "op": "chunk", "b": 64, "chunks": 0, "chunk": 1, "shortest": 200,
         "longest": 8192, "page": 16, "h": 32, "h_kv": 8, "d": 128, "dtype": "bf16", "lens": 7},
        # chunked prefill beside decoding: two requests bring 512 tokens each, the others one
        {"name": "chunk mixed", "op": "chunk", "b": 16, "chunks": 2, "chunk": 512, "shortest": 700,
         "longest": 16384, "page": 64, "h": 32, "h_kv": 8, "d": 128, "dtype": "bf16", "lens": 8},
        # the tables of a decode step
        {"name": "plan decode", "op": "plan", "b": 48, "shortest": 1, "longest": 4000, "new": 1, "page": 16,
         "lens": 9},
        # the tables of a step that takes in many prompts
        {"name": "plan prompts", "op": "plan", "b": 700, "shortest": 0, "longest": 2000, "new": 300, "page": 64,
         "lens": 10},
        # the new rows of a decode step
        {"name": "write decode", "op": "write", "tokens": 48, "page": 16, "h_kv": 8, "d": 128, "dtype": "bf16",
         "fused": False},
        # the rows of a prefill batch, slices of one projection
        {"name": "write prompts", "op": "write", "tokens": 16391, "page": 16, "h_kv": 8, "d": 128,
         "dtype": "bf16", "fused": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    h_kv = rng.choice([1, 2, 3, 4, 8])
    return h_kv * rng.choice([1, 2, 3, 4, 5, 8]), h_kv


def draw(rng):
    op = rng.choice(["prompt", "prompt", "train", "train", "chunk", "chunk", "chunk", "plan", "write"])
    lens = rng.randrange(1 << 30)
    dtype = rng.choice(["bf16", "fp16"])
    if op in ("prompt", "train"):
        longest = _log(rng, 1, 8192 if op == "prompt" else 4096)
        # at most 16384 (prompt) or 8192 (train) tokens, and scores that fit beside the other states
        b = max(1, min(_log(rng, 1, 64), (16384 if op == "prompt" else 8192) // longest,
                       (1 << 27) // longest ** 2))
        h, h_kv = _heads(rng)
        h, h_kv = (h, h_kv) if h <= 32 else (32, 8)
        return {"op": op, "b": b, "shortest": rng.randint(0, longest), "longest": longest, "h": h, "h_kv": h_kv,
                "d": rng.choice([16, 32, 64, 128]), "dtype": dtype, "causal": rng.random() < 0.8,
                "fused": rng.random() < 0.5, "lens": lens}
    if op == "chunk":
        h, h_kv = _heads(rng)
        h, h_kv = (h, h_kv) if h <= 32 else (32, 8)
        longest = _log(rng, 1, 16384)
        chunk = rng.choice([1, 1, rng.randint(2, 8), _log(rng, 9, 512)])
        # gathered caches of at most 512 Ki keys, scores of at most 4 Gi values
        b = max(1, min(_log(rng, 1, 128), (1 << 19) // longest, (1 << 32) // (longest * h * chunk)))
        return {"op": op, "b": b, "chunks": rng.randint(0, b), "chunk": chunk,
                "shortest": rng.randint(0, longest), "longest": longest, "page": rng.choice([16, 32, 64, 128]),
                "h": h, "h_kv": h_kv, "d": rng.choice([16, 32, 64, 128]), "dtype": dtype, "lens": lens}
    if op == "plan":
        b = _log(rng, 1, 1500)
        return {"op": op, "b": b, "shortest": 0, "longest": _log(rng, 1, 4000), "new": _log(rng, 1, 300),
                "page": rng.choice([16, 32, 64, 128]), "lens": lens}
    return {"op": op, "tokens": _log(rng, 1, 16384), "page": rng.choice([16, 32, 64, 128]),
            "h_kv": rng.choice([1, 2, 4, 8]), "d": rng.choice([16, 32, 64, 128]), "dtype": dtype,
            "fused": rng.random() < 0.5}


def _lengths(case):
    """Keys of each sequence: spread between the shortest and the longest, which both occur."""
    r = random.Random(case["lens"])
    n = [r.randint(case["shortest"], case["longest"]) for _ in range(case["b"])]
    n[r.randrange(len(n))] = case["longest"]
    return n


def _chunk_lengths(case):
    """(new tokens, keys with them) of each request of a chunk case; a request has at least its new tokens."""
    keys = _lengths(case)
    new = [case["chunk"] if i < case["chunks"] else 1 for i in range(case["b"])]
    random.Random(case["lens"] + 1).shuffle(new)
    return new, [max(k, n) for k, n in zip(keys, new)]


def _plan_lengths(case):
    """(keys in the cache, new tokens) of each request of a plan case; some requests wait and bring none."""
    r = random.Random(case["lens"])
    old = [r.randint(case["shortest"], case["longest"]) for _ in range(case["b"])]
    new = [case["new"] if case["new"] == 1 else r.randint(0, case["new"]) for _ in range(case["b"])]
    return old, new


def _pages(n, page):
    return -(-n // page)


def _starts(lengths):
    at = [0]
    for n in lengths:
        at.append(at[-1] + n)
    return at


def _pairs(sq, sk, causal):
    """Visible (row, key) pairs of sq rows, the last sq positions of sk keys when causal."""
    if not causal:
        return sq * sk
    return sum(range(max(1, sk - sq + 1), sk + 1))


def work(case):
    op = case["op"]
    if op == "plan":
        old, new = _plan_lengths(case)
        taken = sum(_pages(o + n, case["page"]) - _pages(o, case["page"]) for o, n in zip(old, new))
        # lengths in; starts, lengths and the slot of each token out; each page taken is read and put in the table
        return {"bytes": 4.0 * (4 * case["b"] + 3) + 8.0 * sum(new) + 8.0 * taken, "flops": 0.0}
    if op == "write":
        return {"bytes": case["tokens"] * (8.0 * case["h_kv"] * case["d"] + 8.0), "flops": 0.0}
    h, h_kv, d = case["h"], case["h_kv"], case["d"]
    if op == "chunk":
        new, keys = _chunk_lengths(case)
        pairs = sum(_pairs(n, k, True) for n, k in zip(new, keys))
        pages = sum(_pages(k, case["page"]) for k in keys)
        return {"bytes": 4.0 * sum(new) * h * d + 4.0 * sum(new) * h + 4.0 * sum(keys) * h_kv * d + 4.0 * pages +
                8.0 * case["b"], "flops": 4.0 * pairs * h * d}
    lens = _lengths(case)
    t = sum(lens)
    pairs = sum(_pairs(n, n, case["causal"]) for n in lens)
    out = {"bytes": 4.0 * t * (h + h_kv) * d + 4.0 * t * h, "flops": 4.0 * pairs * h * d}
    if op == "train":  # dO in, dQ, dK and dV out, and five more products
        out["bytes"] += 2.0 * t * (2 * h + 2 * h_kv) * d
        out["flops"] += 10.0 * pairs * h * d
    return out


# ---------------------------------------------------------------- inputs
def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _qkv(g, t, h, h_kv, d, dtype, fused):
    """q [t, h, d], k and v [t, h_kv, d]: slices of one projection's rows, or tensors of their own."""
    if fused:
        x = torch.randn((t, (h + 2 * h_kv) * d), generator=g, device="cuda", dtype=torch.float32).to(dtype)
        q, k, v = x.split((h * d, h_kv * d, h_kv * d), dim=1)
        return q.unflatten(1, (h, d)), k.unflatten(1, (h_kv, d)), v.unflatten(1, (h_kv, d))
    return tuple(torch.randn((t, n, d), generator=g, device="cuda", dtype=torch.float32).to(dtype)
                 for n in (h, h_kv, h_kv))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": dict(case)}
    op = case["op"]
    if op == "plan":
        old, new = _plan_lengths(case)
        page = case["page"]
        have = [_pages(o, page) for o in old]
        want = [_pages(o + n, page) for o, n in zip(old, new)]
        width, used, taken = max(max(want), 1), sum(have), sum(want) - sum(have)
        ids = torch.randperm(used + taken + 17, generator=g, device="cuda").to(torch.int32)
        p = torch.arange(width, device="cuda")[None, :]
        first = _ints(_starts(have)[:-1], torch.int64)[:, None]
        at = (first + p).clamp(max=ids.numel() - 1)
        s["block_table"] = torch.where(p < _ints(have)[:, None], ids[at], -1).contiguous()
        s["free_pages"] = torch.cat([ids[used:], ids[:used]])
        s["free_count"] = _ints([taken + 17])
        s["seqlens"], s["new_lens"] = _ints(old), _ints(new)
        t = sum(new) + 5  # a step's buffers are as long as the longest step's: some entries stay unused
        s["out"] = (torch.empty(case["b"] + 1, dtype=torch.int32, device="cuda"), torch.empty_like(s["seqlens"]),
                    torch.empty(t, dtype=torch.int64, device="cuda"), torch.empty_like(s["free_count"]))
        return s
    dtype, h_kv, d = _DTYPES[case["dtype"]], case["h_kv"], case["d"]
    if op == "write":
        t, page = case["tokens"], case["page"]
        pool = _pages(t, page) + 3
        shape = (pool, page, h_kv, d)
        s["k_pages"], s["v_pages"] = (torch.randn(shape, generator=g, device="cuda").to(dtype) for _ in "kv")
        _, s["k"], s["v"] = _qkv(g, t, h_kv, h_kv, d, dtype, case["fused"])
        slots = torch.randperm(pool * page, generator=g, device="cuda")[:t]
        if t > 4:
            slots[t // 2] = -1  # a padding row of the batch
        s["slots"] = slots
        return s
    h = case["h"]
    s["scale"] = 1.0 / math.sqrt(d)
    if op == "chunk":
        new, keys = _chunk_lengths(case)
        page = case["page"]
        n = [_pages(k, page) for k in keys]
        width, total = max(n) + 2, sum(n)
        ids = torch.randperm(total + 3, generator=g, device="cuda").to(torch.int32)
        p = torch.arange(width, device="cuda")[None, :]
        at = (_ints(_starts(n)[:-1], torch.int64)[:, None] + p).clamp(max=ids.numel() - 1)
        s["block_table"] = torch.where(p < _ints(n)[:, None], ids[at], -1).contiguous()
        s["k_pages"], s["v_pages"] = (torch.randn((total + 3, page, h_kv, d), generator=g, device="cuda",
                                                  dtype=torch.float32).to(dtype) for _ in "kv")
        s["q"] = torch.randn((sum(new), h, d), generator=g, device="cuda").to(dtype)
        s["cu_q"], s["seqlens"] = _ints(_starts(new)), _ints(keys)
        s["max_q"], s["max_k"] = max(new), max(keys)
    else:
        lens = _lengths(case)
        t = sum(lens)
        s["q"], s["k"], s["v"] = _qkv(g, t, h, h_kv, d, dtype, case["fused"])
        s["cu_q"] = _ints(_starts(lens))
        s["max_q"] = s["max_k"] = max(lens)
        if op == "train":
            s["dout"] = torch.randn((t, h, d), generator=g, device="cuda").to(dtype)
            s["grads"] = tuple(torch.empty(x.shape, dtype=dtype, device="cuda") for x in (s["q"], s["k"], s["v"]))
    t = s["q"].shape[0]
    s["o"] = torch.empty((t, h, d), dtype=dtype, device="cuda")
    s["lse"] = torch.empty((h, t), dtype=torch.float32, device="cuda")
    return s


# ---------------------------------------------------------------- one pass
def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        return _own(state, c, op)
    if op == "plan":
        return _plain_plan(state, c["page"])
    if op == "write":
        return _plain_write(state)
    return _plain_attention(state, c, op)


def _own(s, c, op):
    import exact_attention_65_gb300 as ea

    if op == "plan":
        cu, lens, slots, left = s["out"]
        ea.attn_paged_plan(s["seqlens"], s["new_lens"], s["block_table"], s["free_pages"], s["free_count"],
                           c["page"], cu_seqlens_q=cu, seqlens_out=lens, slot_map=slots, free_left=left)
        return s["block_table"], cu, lens, slots, left
    if op == "write":
        ea.attn_paged_write(s["k"], s["v"], s["slots"], s["k_pages"], s["v_pages"])
        return s["k_pages"], s["v_pages"]
    if op == "chunk":
        return ea.attn_chunk_paged(s["q"], s["k_pages"], s["v_pages"], s["block_table"], s["cu_q"], s["seqlens"],
                                   max_seqlen_q=s["max_q"], out=s["o"], lse=s["lse"], causal=True)
    o, lse = ea.attn_fwd_packed(s["q"], s["k"], s["v"], s["cu_q"], s["cu_q"], max_seqlen_q=s["max_q"],
                                out=s["o"], lse=s["lse"], causal=c["causal"])
    if op == "prompt":
        return o, lse
    dq, dk, dv = s["grads"]
    ea.attn_bwd_packed(s["q"], s["k"], s["v"], o, lse, s["dout"], s["cu_q"], s["cu_q"],
                       dq=dq, dk=dk, dv=dv, causal=c["causal"])
    return o, lse, dq, dk, dv


def _plain_plan(s, page):
    old, new, table = s["seqlens"].long(), s["new_lens"].long(), s["block_table"]
    width = table.shape[1]
    have = (old + page - 1) // page
    want = ((old + new + page - 1) // page).clamp(max=width)
    need = (want - have).clamp(min=0)
    base = need.cumsum(0) - need
    p = torch.arange(width, device=table.device)[None, :]
    k = p - have[:, None]
    at = s["free_count"].long() - 1 - (base[:, None] + k)
    page_of = torch.where(at >= 0, s["free_pages"][at.clamp(0, s["free_pages"].numel() - 1)], -1)
    table = torch.where((k >= 0) & (p < want[:, None]), page_of, table)
    ends = new.cumsum(0)
    cu = torch.cat([torch.zeros_like(ends[:1]), ends])
    t = torch.arange(s["out"][2].numel(), device=table.device)
    i = torch.searchsorted(ends, t, right=True)
    there = i < old.numel()
    i = i.clamp(max=old.numel() - 1)
    pos = old[i] + t - cu[i]
    pg = table[i, (pos // page).clamp(max=width - 1)].long()
    slots = torch.where(there & (pg >= 0) & (pos < width * page), pg * page + pos % page, -1)
    return (table, cu.int(), torch.minimum(old + new, torch.full_like(old, width * page)).int(), slots,
            (s["free_count"].long() - need.sum()).int())


def _plain_write(s):
    out = []
    keep = s["slots"] >= 0
    at = s["slots"][keep]
    for new, pool in ((s["k"], s["k_pages"]), (s["v"], s["v_pages"])):
        pool.view(-1, pool.shape[2], pool.shape[3])[at] = new[keep]
        out.append(pool)
    return tuple(out)


def _plain_attention(s, c, op):
    """Sequences padded to the longest, every score kept: [b, h_kv, group, rows, keys]."""
    q, scale, h, h_kv, d = s["q"], s["scale"], c["h"], c["h_kv"], c["d"]
    cu = s["cu_q"].long()
    sq = cu[1:] - cu[:-1]
    sk = s["seqlens"].long() if op == "chunk" else sq
    causal = op == "chunk" or c["causal"]
    r = torch.arange(s["max_q"], device="cuda")
    j = torch.arange(s["max_k"], device="cuda")
    rows = (cu[:-1, None] + r).clamp(max=q.shape[0] - 1)
    has_row, has_key = r < sq[:, None], j < sk[:, None]
    if op == "chunk":
        page = c["page"]
        pages = s["block_table"][:, : -(-s["max_k"] // page)].clamp(min=0).long()
        kk, vv = (x[pages].flatten(1, 2)[:, : s["max_k"]].float() for x in (s["k_pages"], s["v_pages"]))
    else:
        keys = (cu[:-1, None] + j).clamp(max=q.shape[0] - 1)
        kk, vv = s["k"][keys].float(), s["v"][keys].float()
    kk, vv = (torch.where(has_key[:, :, None, None], x, 0.0).permute(0, 2, 3, 1)[:, :, None] for x in (kk, vv))

    def grouped(x):  # [tokens, h, d] -> [b, h_kv, group, rows, d]
        x = torch.where(has_row[:, :, None, None], x[rows].float(), 0.0)
        return x.unflatten(2, (h_kv, h // h_kv)).permute(0, 2, 3, 1, 4)

    qq = grouped(q)
    sees = has_row[:, :, None] & has_key[:, None, :]
    if causal:
        sees = sees & (j <= r[None, :, None] + (sk - sq)[:, None, None])
    sees = sees[:, None, None]
    score = torch.where(sees, torch.matmul(qq, kk) * scale, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score.sub_(top))
    total = p.sum(-1, keepdim=True)
    lse = torch.where(total > 0, top + torch.log(total), -math.inf)
    p = p / torch.where(total > 0, total, 1.0)
    oo = torch.matmul(p, vv.transpose(-1, -2))

    def packed(x, at, n):  # [b, heads, groups, rows, d] -> [tokens, heads * groups, d]
        return x.permute(0, 3, 1, 2, 4).flatten(2, 3)[at, n]

    token = torch.arange(q.shape[0], device="cuda")
    seq = torch.searchsorted(cu[1:].contiguous(), token, right=True)
    at = token - cu[seq]
    o = packed(oo, seq, at).to(q.dtype)
    lse = packed(lse, seq, at)[:, :, 0].t().contiguous()
    if op != "train":
        return o, lse
    do = grouped(s["dout"])
    dv = torch.matmul(p.transpose(-1, -2), do).sum(2, keepdim=True)
    dp = torch.matmul(do, vv)
    ds = p * (dp - (do * oo).sum(-1, keepdim=True))
    dq = torch.matmul(ds, kk.transpose(-1, -2)) * scale
    dk = torch.matmul(ds.transpose(-1, -2), qq).sum(2, keepdim=True) * scale
    return (o, lse, *(packed(x, seq, at).to(q.dtype) for x in (dq, dk, dv)))


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    """The definition in 64 bits, one sequence and one head at a time."""
    op = case["op"]
    if op == "plan":
        return None  # whole numbers
    s = prepare(case, seed)
    if op == "write":
        pools = []
        slots = s["slots"].tolist()
        rows = [t for t, x in enumerate(slots) if x >= 0]
        there = torch.tensor([slots[t] for t in rows], device="cuda", dtype=torch.int64)
        for x, pool in (("k", "k_pages"), ("v", "v_pages")):
            y = s[pool].double().flatten(0, 1)
            y[there] = s[x].double()[torch.tensor(rows, device="cuda", dtype=torch.int64)]
            pools.append(y.reshape(s[pool].shape))
        return tuple(pools)
    h, h_kv, d = case["h"], case["h_kv"], case["d"]
    if op == "chunk":
        new, keys = _chunk_lengths(case)
    else:
        new = keys = _lengths(case)
    causal = op == "chunk" or case["causal"]
    starts = _starts(new)
    f64 = {"dtype": torch.float64, "device": "cuda"}
    t = starts[-1]
    o, lse = torch.zeros((t, h, d), **f64), torch.full((h, t), -math.inf, **f64)
    dq, dk, dv = torch.zeros((t, h, d), **f64), torch.zeros((t, h_kv, d), **f64), torch.zeros((t, h_kv, d), **f64)
    for i, (n, m) in enumerate(zip(new, keys)):
        if n == 0 or m == 0:
            continue
        a, z = starts[i], starts[i + 1]
        if op == "chunk":
            ids = s["block_table"][i, : _pages(m, case["page"])].long()
            kk, vv = s["k_pages"][ids].flatten(0, 1)[:m].double(), s["v_pages"][ids].flatten(0, 1)[:m].double()
        else:
            kk, vv = s["k"][a:z].double(), s["v"][a:z].double()
        hidden = torch.ones((n, m), dtype=torch.bool, device="cuda").triu_(m - n + 1) if causal else None
        for x in range(h):
            y = x // (h // h_kv)
            qx = s["q"][a:z, x].double()
            w = (qx @ kk[:, y].t()).mul_(s["scale"])
            if causal:
                w.masked_fill_(hidden, -math.inf)
            lx = torch.logsumexp(w, 1)
            w = w.sub_(lx[:, None]).exp_()
            o[a:z, x], lse[x, a:z] = w @ vv[:, y], lx
            if op == "train":
                gx = s["dout"][a:z, x].double()
                dv[a:z, y] += w.t() @ gx
                e = gx @ vv[:, y].t()
                e = w * (e - (w * e).sum(1, keepdim=True))
                dq[a:z, x] = (e @ kk[:, y]) * s["scale"]
                dk[a:z, y] += (e.t() @ qx) * s["scale"]
    return (o, lse, dq, dk, dv) if op == "train" else (o, lse)
