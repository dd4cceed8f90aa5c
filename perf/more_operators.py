"""Work of the rotating appends and of the 4-bit paged cache, for timing and for comparing outputs.

Four operators, as a serving program calls them:

    append   attn_paged_append: a step's queries and keys rotated by their
             positions, keys and values into 16-bit pages
    append4  attn_paged_append_q4, then attn_paged_read_q4 of the same slots:
             the same into pages of 4 bits, and the rows as the cache holds
             them (what a prompt's own attention reads, so that it sees what
             later steps will see)
    read4    attn_paged_read_q4: rows of a 4-bit cache back in 16 bits, for a
             request that moves
    attend4  attn_chunk_paged_q4: the new tokens of each request (one, or a
             chunk of a prompt) over a 4-bit cache

A 4-bit pool is uint8 [num_pages, h_kv, page_size * 9 d / 16]: a page of a head
holds page_size rows of d / 2 bytes of e2m1 codes (channel 2 i in the low half
of byte i), then page_size rows of d / 16 e4m3 scales, one for 16 channels. A
value is code * scale * the tensor's scale.

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
        # the new token of a single user: the call's own latency
        {"name": "append one", "op": "append", "tokens": 1, "page": 16, "h": 32, "h_kv": 8, "d": 128, "rot": 128,
         "far": 4096, "interleaved": False, "dtype": "bf16", "fused": True},
        # a decode step of a full batch; half of each head turns, in neighbouring pairs
        {"name": "append batch", "op": "append", "tokens": 61, "page": 64, "h": 16, "h_kv": 4, "d": 64, "rot": 32,
         "far": 8192, "interleaved": True, "dtype": "fp16", "fused": False},
        # a prefill step, slices of one projection, positions far into a long context
        {"name": "append prompts", "op": "append", "tokens": 16391, "page": 16, "h": 32, "h_kv": 8, "d": 128,
         "rot": 128, "far": 131072, "interleaved": False, "dtype": "bf16", "fused": True},
        # the same three into 4 bits
        {"name": "append4 one", "op": "append4", "tokens": 1, "page": 16, "h": 32, "h_kv": 8, "d": 128, "rot": 128,
         "far": 4096, "interleaved": False, "dtype": "bf16", "fused": True, "ks": 1.0, "vs": 1.0},
        {"name": "append4 prompts", "op": "append4", "tokens": 16391, "page": 16, "h": 32, "h_kv": 8, "d": 128,
         "rot": 128, "far": 131072, "interleaved": False, "dtype": "bf16", "fused": True, "ks": 1.0, "vs": 0.125},
        # one request's cache moves to another pool
        {"name": "read4 request", "op": "read4", "tokens": 777, "page": 16, "h_kv": 8, "d": 128, "dtype": "bf16",
         "ks": 1.0, "vs": 1.0},
        # the requests of a whole machine move; a tensor scale that is no power of two
        {"name": "read4 batch", "op": "read4", "tokens": 40001, "page": 64, "h_kv": 8, "d": 128, "dtype": "fp16",
         "ks": 0.37, "vs": 0.21},
        # one user, one new token: latency
        {"name": "attend4 one", "op": "attend4", "b": 1, "chunks": 0, "chunk": 1, "shortest": 900, "longest": 900,
         "page": 16, "h": 32, "h_kv": 8, "d": 128, "dtype": "bf16", "ks": 1.0, "vs": 1.0, "lens": 6},
        # a full decode batch, one token each, caches of very different lengths
        {"name": "attend4 batch", "op": "attend4", "b": 64, "chunks": 0, "chunk": 1, "shortest": 200,
         "longest": 8192, "page": 16, "h": 32, "h_kv": 8, "d": 128, "dtype": "bf16", "ks": 1.0, "vs": 1.0, "lens": 7},
        # two users deep into a long context, a token and three drafts of it each, every head dim of 64
        {"name": "attend4 long", "op": "attend4", "b": 2, "chunks": 2, "chunk": 4, "shortest": 90001,
         "longest": 131072, "page": 64, "h": 16, "h_kv": 4, "d": 64, "dtype": "fp16", "ks": 0.5, "vs": 0.25,
         "lens": 9},
        # chunked prefill beside decoding: two requests bring 512 tokens each, the others one
        {"name": "attend4 mixed", "op": "attend4", "b": 16, "chunks": 2, "chunk": 512, "shortest": 700,
         "longest": 16384, "page": 64, "h": 32, "h_kv": 8, "d": 128, "dtype": "bf16", "ks": 1.0, "vs": 1.0,
         "lens": 8},
        # whole prompts through the cache
        {"name": "attend4 prompts", "op": "attend4", "b": 5, "chunks": 5, "chunk": 1900, "shortest": 1900,
         "longest": 2100, "page": 16, "h": 32, "h_kv": 8, "d": 128, "dtype": "bf16", "ks": 1.0, "vs": 1.0,
         "lens": 10},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    h_kv = rng.choice([1, 2, 3, 4, 8])
    h = h_kv * rng.choice([1, 2, 3, 4, 5, 8])
    return (h, h_kv) if h <= 32 else (32, 8)


def draw(rng):
    op = rng.choice(["append", "append", "append4", "append4", "read4", "attend4", "attend4", "attend4", "attend4"])
    h, h_kv = _heads(rng)
    d = rng.choice([16, 32, 64, 128])
    case = {"op": op, "page": rng.choice([16, 32, 48, 64, 128]), "h_kv": h_kv, "d": d,
            "dtype": rng.choice(["bf16", "fp16"])}
    if op != "append":
        case.update(ks=rng.choice([1.0, 0.5, 0.37]), vs=rng.choice([1.0, 0.125, 0.21]))
    if op in ("append", "append4"):
        case.update(tokens=_log(rng, 1, 16384), h=h, rot=16 * rng.randint(1, d // 16), far=_log(rng, 100, 131072),
                    interleaved=rng.random() < 0.4, fused=rng.random() < 0.5)
    elif op == "read4":
        case.update(tokens=_log(rng, 1, 40000))
    else:
        longest = _log(rng, 1, 131072)
        chunk = rng.choice([1, 1, rng.randint(2, 8), _log(rng, 9, 2048)])
        # gathered caches of at most 256 Ki keys, scores of at most 2 Gi values
        b = max(1, min(_log(rng, 1, 128), (1 << 18) // longest, (1 << 31) // (longest * h * chunk)))
        chunk = max(1, min(chunk, (1 << 31) // (longest * h * b)))
        case.update(b=b, chunks=rng.randint(0, b), chunk=chunk, shortest=rng.randint(0, longest), longest=longest,
                    h=h, lens=rng.randrange(1 << 30))
        while work(case)["flops"] > 1.6e11:
            case["chunk"] = case["chunk"] // 2
    return case


def _lengths(case):
    """(new tokens, keys with them) of each request: keys between the shortest
    and the longest, which both occur; a request has at least its new tokens."""
    r = random.Random(case["lens"])
    keys = [r.randint(case["shortest"], case["longest"]) for _ in range(case["b"])]
    keys[r.randrange(len(keys))] = case["longest"]
    new = [case["chunk"] if i < case["chunks"] else 1 for i in range(case["b"])]
    r.shuffle(new)
    return new, [max(k, n) for k, n in zip(keys, new)]


def _pages(n, page):
    return -(-n // page)


def _starts(lengths):
    at = [0]
    for n in lengths:
        at.append(at[-1] + n)
    return at


def work(case):
    op, h_kv, d = case["op"], case["h_kv"], case["d"]
    row = h_kv * d  # values of a token's keys
    if op == "attend4":
        h = case["h"]
        new, keys = _lengths(case)
        pairs = sum(sum(range(max(1, k - n + 1), k + 1)) for n, k in zip(new, keys))
        pages = sum(_pages(k, case["page"]) for k in keys)
        return {"bytes": 4.0 * sum(new) * h * d + 4.0 * sum(new) * h + 2 * 0.5625 * sum(keys) * row + 4.0 * pages +
                8.0 * case["b"], "flops": 4.0 * pairs * h * d}
    t = case["tokens"]
    if op == "read4":
        return {"bytes": t * (2 * 0.5625 * row + 4.0 * row + 8.0), "flops": 4.0 * t * row}
    h = case["h"]
    # q in and out, k and v in, a row of the table, position and slot; pages out (4 bits: and the rows read back)
    out = 4.0 * row if op == "append" else 2 * 0.5625 * row + 4.0 * row
    return {"bytes": t * (4.0 * h * d + 4.0 * row + 4.0 * case["rot"] + 16.0 + out),
            "flops": 3.0 * t * (h + h_kv) * case["rot"] + (0.0 if op == "append" else 6.0 * t * row)}


# ---------------------------------------------------------------- the 4-bit format
def _quantised(x, scale):
    """Codes (0 .. 15) and e4m3 scales (as bytes) of x [..., d], fp32: 16
    neighbours share s = amax / (6 scale), a code is x / (s scale), each to the
    nearest, ties to even. A group that holds an infinity or a NaN gets the
    scale NaN."""
    g = x.unflatten(-1, (-1, 16))
    amax = g.abs().amax(-1, keepdim=True)
    s = (amax / torch.full_like(amax, 6.0 * scale)).clamp(max=448.0)
    s = torch.where(torch.isfinite(amax), s, math.nan).to(torch.float8_e4m3fn)
    unit = s.float() * scale
    y = torch.where(unit > 0, g / unit, 0.0)
    a = y.abs().clamp(max=6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = torch.round(a / step) * step
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = torch.where(torch.signbit(y), code + 8, code)
    return code.flatten(-2), s.squeeze(-1).view(torch.uint8)


def _to_bytes(code, s, pool, page, slots):
    """Rows [t, h_kv, d] of codes and [t, h_kv, d / 16] of scales into the pool's slots."""
    d = code.shape[-1]
    codes, scales = _parts(pool, page, d)
    both = code[..., 0::2] + 16 * code[..., 1::2]
    codes[slots // page, :, slots % page] = both
    scales[slots // page, :, slots % page] = s


def _parts(pool, page, d):
    """Views of a pool's codes [num_pages, h_kv, page, d / 2] and scales [num_pages, h_kv, page, d / 16]."""
    return pool[..., : page * d // 2].unflatten(-1, (page, d // 2)), \
        pool[..., page * d // 2:].unflatten(-1, (page, d // 16))


def _values(pool, page, d, pages, rows, scale):
    """Values [..., h_kv, d] in fp32 of the pool's given pages and rows in them."""
    codes, scales = _parts(pool, page, d)
    both = codes[pages, :, rows].to(torch.int64)
    code = torch.stack((both & 15, both >> 4), -1).flatten(-2)
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=pool.device)
    table = torch.cat([table, -table])
    s = scales[pages, :, rows].view(torch.float8_e4m3fn).float() * scale
    return (table[code].unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)


# ---------------------------------------------------------------- inputs
def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _pool(g, pages, page, h_kv, d, scale):
    """A pool whose every row holds the values of some token."""
    pool = torch.empty((pages, h_kv, page * 9 * d // 16), dtype=torch.uint8, device="cuda")
    per = max(1, (1 << 26) // (page * h_kv * d))
    for at in range(0, pages, per):
        n = min(per, pages - at)
        code, s = _quantised(_randn(g, n * page, h_kv, d), scale)
        _to_bytes(code, s, pool, page, torch.arange(at * page, (at + n) * page, device="cuda"))
    return pool


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": dict(case)}
    op, page, h_kv, d = case["op"], case["page"], case["h_kv"], case["d"]
    dtype = _DTYPES[case["dtype"]]
    if op == "attend4":
        h = case["h"]
        new, keys = _lengths(case)
        n = [_pages(k, page) for k in keys]
        width, total = max(n) + 2, sum(n)
        ids = torch.randperm(total + 3, generator=g, device="cuda").to(torch.int32)
        p = torch.arange(width, device="cuda")[None, :]
        at = (_ints(_starts(n)[:-1], torch.int64)[:, None] + p).clamp(max=ids.numel() - 1)
        s["block_table"] = torch.where(p < _ints(n)[:, None], ids[at], -1).contiguous()
        s["k_pages"] = _pool(g, total + 3, page, h_kv, d, case["ks"])
        s["v_pages"] = _pool(g, total + 3, page, h_kv, d, case["vs"])
        s["q"] = _randn(g, sum(new), h, d).to(dtype)
        s["cu_q"], s["seqlens"] = _ints(_starts(new)), _ints(keys)
        s["max_q"], s["max_k"] = max(new), max(keys)
        s["scale"] = 1.0 / math.sqrt(d)
        s["o"] = torch.empty((sum(new), h, d), dtype=dtype, device="cuda")
        s["lse"] = torch.empty((h, sum(new)), dtype=torch.float32, device="cuda")
        return s
    t = case["tokens"]
    pages = _pages(t, page) + 3
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:t]
    if t > 4:
        slots[t // 2] = -1  # a padding row of the batch
    s["slots"] = slots
    if op == "append":
        s["k_pages"], s["v_pages"] = (_randn(g, pages, page, h_kv, d).to(dtype) for _ in "kv")
    else:
        s["k_pages"] = _pool(g, pages, page, h_kv, d, case["ks"])
        s["v_pages"] = _pool(g, pages, page, h_kv, d, case["vs"])
        s["rows"] = tuple(torch.empty((t, h_kv, d), dtype=dtype, device="cuda") for _ in "kv")
    if op == "read4":
        return s
    h, rot = case["h"], case["rot"]
    if case["fused"]:
        x = _randn(g, t, (h + 2 * h_kv) * d).to(dtype)
        s["q"], s["k"], s["v"] = (y.unflatten(1, (-1, d)) for y in x.split((h * d, h_kv * d, h_kv * d), dim=1))
    else:
        s["q"], s["k"], s["v"] = (_randn(g, t, n, d).to(dtype) for n in (h, h_kv, h_kv))
    # the angles of every position, cosines and then sines of each
    turn = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    angle = torch.arange(case["far"], device="cuda", dtype=torch.float64)[:, None] * turn
    s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    s["positions"] = torch.randint(0, case["far"], (t,), generator=g, device="cuda")
    s["q_out"] = torch.empty((t, h, d), dtype=dtype, device="cuda")
    return s


# ---------------------------------------------------------------- one pass
def run(state):
    c = state["case"]
    if own:
        return _own(state, c, c["op"])
    if c["op"] == "attend4":
        return _plain_attend(state, c)
    if c["op"] == "read4":
        return _plain_read(state, c)
    return _plain_append(state, c)


def _own(s, c, op):
    import exact_attention_65_gb300 as ea

    if op == "attend4":
        return ea.attn_chunk_paged_q4(s["q"], s["k_pages"], s["v_pages"], s["block_table"], s["cu_q"], s["seqlens"],
                                      max_seqlen_q=s["max_q"], k_scale=c["ks"], v_scale=c["vs"], out=s["o"],
                                      lse=s["lse"], causal=True)
    if op == "append":
        q = ea.attn_paged_append(s["q"], s["k"], s["v"], s["cos_sin"], s["positions"], s["slots"], s["k_pages"],
                                 s["v_pages"], q_out=s["q_out"], interleaved=c["interleaved"])
        return q, s["k_pages"], s["v_pages"]
    q = ()
    if op == "append4":
        q = (ea.attn_paged_append_q4(s["q"], s["k"], s["v"], s["cos_sin"], s["positions"], s["slots"], s["k_pages"],
                                     s["v_pages"], k_scale=c["ks"], v_scale=c["vs"], q_out=s["q_out"],
                                     interleaved=c["interleaved"]),)
    return *q, *ea.attn_paged_read_q4(s["k_pages"], s["v_pages"], s["slots"], c["d"], k_scale=c["ks"],
                                      v_scale=c["vs"], k=s["rows"][0], v=s["rows"][1])


def _rotated(x, cos_sin, positions, interleaved):
    """x [t, heads, d] in fp32 with its first rot channels turned in pairs."""
    rot = cos_sin.shape[1]
    cos, sin = cos_sin[positions][:, None].split(rot // 2, -1)
    y, rest = x[..., :rot].float(), x[..., rot:].float()
    a, b = (y[..., 0::2], y[..., 1::2]) if interleaved else y.split(rot // 2, -1)
    pair = (a * cos - b * sin, b * cos + a * sin)
    y = torch.stack(pair, -1).flatten(-2) if interleaved else torch.cat(pair, -1)
    return torch.cat([y, rest], -1)


def _plain_append(s, c):
    turn = (s["cos_sin"], s["positions"], c["interleaved"])
    q = _rotated(s["q"], *turn).to(s["q"].dtype)
    k, v, page = _rotated(s["k"], *turn), s["v"].float(), c["page"]
    keep = s["slots"] >= 0
    at = s["slots"][keep]
    if c["op"] == "append":
        s["k_pages"][at // page, at % page] = k[keep].to(q.dtype)
        s["v_pages"][at // page, at % page] = s["v"][keep]
        return q, s["k_pages"], s["v_pages"]
    _to_bytes(*_quantised(k[keep], c["ks"]), s["k_pages"], page, at)
    _to_bytes(*_quantised(v[keep], c["vs"]), s["v_pages"], page, at)
    return q, *_plain_read(s, c)


def _plain_read(s, c):
    page, dtype, slots = c["page"], _DTYPES[c["dtype"]], s["slots"]
    there = (slots >= 0)[:, None, None]
    at = slots.clamp(min=0)
    k = _values(s["k_pages"], page, c["d"], at // page, at % page, c["ks"])
    v = _values(s["v_pages"], page, c["d"], at // page, at % page, c["vs"])
    return torch.where(there, k, 0.0).to(dtype), torch.where(there, v, 0.0).to(dtype)


def _plain_attend(s, c):
    """Requests padded to the longest, every score kept: [b, h_kv, group, rows, keys]."""
    q, h, h_kv, d, page = s["q"], c["h"], c["h_kv"], c["d"], c["page"]
    cu, sk = s["cu_q"].long(), s["seqlens"].long()
    sq = cu[1:] - cu[:-1]
    r = torch.arange(s["max_q"], device=q.device)
    j = torch.arange(s["max_k"], device=q.device)
    rows = (cu[:-1, None] + r).clamp(max=q.shape[0] - 1)
    has_row, has_key = r < sq[:, None], j < sk[:, None]
    pages = s["block_table"].clamp(min=0).long()[:, j // page]
    at = (j % page).expand_as(pages)
    kk = _values(s["k_pages"], page, d, pages, at, c["ks"])
    vv = _values(s["v_pages"], page, d, pages, at, c["vs"])
    kk = torch.where(has_key[:, :, None, None], kk, 0.0).permute(0, 2, 3, 1)[:, :, None]
    vv = torch.where(has_key[:, :, None, None], vv, 0.0).permute(0, 2, 1, 3)[:, :, None]
    qq = torch.where(has_row[:, :, None, None], q[rows].float(), 0.0)
    qq = qq.unflatten(2, (h_kv, h // h_kv)).permute(0, 2, 3, 1, 4)
    sees = has_row[:, :, None] & has_key[:, None, :] & (j <= r[None, :, None] + (sk - sq)[:, None, None])
    sees = sees[:, None, None]
    score = torch.where(sees, torch.matmul(qq, kk) * s["scale"], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score.sub_(top))
    total = p.sum(-1, keepdim=True)
    lse = torch.where(total > 0, top + torch.log(total), -math.inf)
    o = torch.matmul(p, vv) / torch.where(total > 0, total, 1.0)
    token = torch.arange(q.shape[0], device=q.device)
    seq = torch.searchsorted(cu[1:].contiguous(), token, right=True)
    n = token - cu[seq]
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[seq, n].to(q.dtype)
    return o, lse.permute(0, 3, 1, 2, 4).flatten(2, 3)[seq, n][:, :, 0].t().contiguous()


# ---------------------------------------------------------------- 64 bits
_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _exact_rows(x, scale):
    """What the 4-bit cache holds of x [t, heads, d] (64 bits), by comparing with the borders between values."""
    g = x.reshape(*x.shape[:-1], -1, 16)
    s = g.abs().amax(-1, keepdim=True) / (6.0 * scale)
    # the e4m3 value nearest to s: a multiple of 2^(e - 3), of 2^-9 at least
    e = torch.frexp(s.clamp(max=448.0, min=2.0 ** -6))[1].double() - 1
    quantum = torch.exp2(e - 3)
    s = torch.round(s.clamp(max=448.0) / quantum) * quantum
    y = torch.where(s > 0, g / torch.where(s > 0, s * scale, 1.0), 0.0)
    a, value = y.abs(), torch.zeros_like(y)
    for i in range(1, 8):
        border = (_GRID[i - 1] + _GRID[i]) / 2
        # a tie goes to the neighbour whose code is even
        value = torch.where(a >= border if i % 2 == 0 else a > border, _GRID[i], value)
    return (torch.sign(y) * value * s * scale).reshape(x.shape)


def _exact_values(pool, ids, page, d, scale):
    """Values [len(ids) * page, h_kv, d] of whole pages, in 64 bits."""
    raw = pool[ids]
    both = raw[..., : page * d // 2].reshape(len(ids), -1, page, d // 2).permute(0, 2, 1, 3).flatten(0, 1).long()
    s = raw[..., page * d // 2:].reshape(len(ids), -1, page, d // 16).permute(0, 2, 1, 3).flatten(0, 1).long()
    grid = torch.tensor(_GRID, dtype=torch.float64, device=pool.device)
    out = torch.empty((*both.shape[:2], d), dtype=torch.float64, device=pool.device)
    for half, nibble in enumerate((both & 15, both >> 4)):
        out[..., half::2] = grid[nibble & 7] * (1 - 2 * (nibble >> 3))
    e, m = s >> 3 & 15, (s & 7).double()
    s = torch.where(e > 0, (1 + m / 8) * torch.exp2(e.double() - 7), m * 2.0 ** -9)
    return out * s.repeat_interleave(16, -1) * scale


def exact(case, seed):
    """The definition in 64 bits; attention one request and one head at a time."""
    s = prepare(case, seed)
    op, page, h_kv, d = case["op"], case["page"], case["h_kv"], case["d"]
    if op == "attend4":
        h = case["h"]
        new, keys = _lengths(case)
        at = _starts(new)
        o = torch.zeros((at[-1], h, d), dtype=torch.float64, device="cuda")
        lse = torch.full((h, at[-1]), -math.inf, dtype=torch.float64, device="cuda")
        for i, (n, m) in enumerate(zip(new, keys)):
            if m == 0:
                continue
            ids = s["block_table"][i, : _pages(m, page)].long()
            kk = _exact_values(s["k_pages"], ids, page, d, case["ks"])[:m]
            vv = _exact_values(s["v_pages"], ids, page, d, case["vs"])[:m]
            hidden = torch.ones((n, m), dtype=torch.bool, device="cuda").triu_(m - n + 1)
            for x in range(h):
                y = x // (h // h_kv)
                w = (s["q"][at[i]:at[i + 1], x].double() @ kk[:, y].t()) * s["scale"]
                w = w.masked_fill_(hidden, -math.inf)
                lx = torch.logsumexp(w, 1)
                o[at[i]:at[i + 1], x], lse[x, at[i]:at[i + 1]] = (w - lx[:, None]).exp() @ vv[:, y], lx
        return o, lse
    slots = s["slots"].tolist()
    there = torch.tensor([i for i, x in enumerate(slots) if x >= 0], device="cuda", dtype=torch.int64)
    to = torch.tensor([x for x in slots if x >= 0], device="cuda", dtype=torch.int64)
    if op == "read4":
        rows = []
        for name, scale in (("k_pages", case["ks"]), ("v_pages", case["vs"])):
            ids = torch.arange(s[name].shape[0], device="cuda")
            y = torch.zeros((case["tokens"], h_kv, d), dtype=torch.float64, device="cuda")
            y[there] = _exact_values(s[name], ids, page, d, scale)[to]
            rows.append(y)
        return tuple(rows)
    rot = case["rot"]
    table = s["cos_sin"].double()[s["positions"]]
    # each pair as a complex number times the position's
    turn = torch.complex(table[:, : rot // 2], table[:, rot // 2:])[:, None]

    def rotated(x):
        x = x.double().clone()
        y = x[..., :rot]
        i = torch.arange(rot // 2, device="cuda")
        first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rot // 2)
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return x

    q, k, v = rotated(s["q"]), rotated(s["k"]), s["v"].double()
    if op == "append":
        pools = []
        for x, name in ((k, "k_pages"), (v, "v_pages")):
            pool = s[name].double().flatten(0, 1)
            pool[to] = x[there]
            pools.append(pool.reshape(s[name].shape))
        return q, *pools
    rows = []
    for x, scale in ((k, case["ks"]), (v, case["vs"])):
        y = torch.zeros_like(x)
        y[there] = _exact_rows(x, scale)[there]
        rows.append(y)
    return q, *rows
