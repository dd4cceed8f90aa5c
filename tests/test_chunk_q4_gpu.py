"""Chunks of new tokens over a cache held in 4 bits (attn_chunk_paged_q4)
against the fp64 oracle over the values that the cache holds, and a serving
loop of plan, append and attention.

Bounds as in packed_parity: what enters the products is exact, P is rounded to
fp16 whatever the type (half a step of the type covers it), O once. Values of P
below 2^-24 of fp16's smallest are lost: 2^-31 of the row's largest at most, per
key, and 2^-30 with its rounding.
"""
import numpy as np
import pytest
import torch

from packed_parity import default_scale, fp32_slack, starts, unit_roundoff

pytestmark = pytest.mark.gpu


def ints(x, dtype=torch.int32):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


def make_cache(oracle, lens, h_kv, d, page, ks, vs, seed, spare=3):
    """Shuffled 4-bit pages; rows past each request's end, and spare pages, hold
    scales of NaN; tables whose entries past it are out of range; the values of
    each request's keys in order."""
    r = np.random.default_rng(seed)
    n = [-(-m // page) for m in lens]
    width, pool = max(max(n), 1) + 1, sum(n) + spare
    perm = r.permutation(pool).tolist()
    table = np.array([[-1, 10 ** 6, pool][i % 3] for i in range(width)])[None].repeat(len(lens), 0)
    pools, values = [], []
    for i in range(len(lens)):
        table[i, :n[i]] = [perm.pop() for _ in range(n[i])]
    slots = np.concatenate([table[i, np.arange(m) // page] * page + np.arange(m) % page
                            for i, m in enumerate(lens)]).astype(np.int64)
    for scale in (ks, vs):
        code = r.integers(0, 256, (pool * page, h_kv, d)).astype(np.uint8)
        s = np.full((pool * page, h_kv, d // 16), 127, dtype=np.uint8)
        code[slots], s[slots] = oracle.q4_quantise(r.standard_normal((len(slots), h_kv, d)), scale)
        code &= 15
        pools.append(torch.from_numpy(oracle.q4_pool(code, s, pool, page)))
        values.append(oracle.q4_values(code[slots], s[slots], float(np.float32(scale))))
    return *pools, torch.tensor(table, dtype=torch.int32), *values


def check(o, lse, q, k, v, cq, ck, causal, dtype, oracle, scale=None):
    d = q.shape[2]
    scale = default_scale(d) if scale is None else scale
    o_ref, l_ref = oracle.packed_attention(q, k, v, cq, ck, scale, causal)
    a_ref, _ = oracle.packed_attention(q, k, np.abs(v), cq, ck, scale, causal)
    rows = int(cq[-1])
    slack = fp32_slack(q, torch.tensor(k), scale, d)
    o64, l64 = o.double().cpu().numpy()[:rows], lse.double().cpu().numpy()[:, :rows]
    o_ref, l_ref, a_ref = o_ref[:rows], l_ref[:, :rows], a_ref[:rows]
    seen = np.isfinite(l_ref)
    assert np.all(np.isneginf(l64[~seen])) and np.all(o64.transpose(1, 0, 2)[~seen] == 0.0)
    assert np.all(np.isfinite(o64)) and np.all(np.isfinite(l64[seen]))
    u = unit_roundoff(dtype)
    # below normal numbers steps have one size; lost values of P, of every key
    lost = 2.0 ** -30 * float(np.diff(ck).max(initial=0)) * float(np.abs(v).max(initial=0.0))
    bound = (u + slack) * (a_ref + np.abs(o_ref)) + torch.finfo(dtype).tiny * u + lost
    err = np.abs(o64 - o_ref)
    assert np.all(err <= bound), f"O off by {err.max():.3e}, {(err - bound).max():.3e} over its bound"
    assert np.abs(l64[seen] - l_ref[seen]).max(initial=0.0) <= slack


def run(ea, oracle, new, lens, h, h_kv, d, page, dtype, causal=True, seed=5, hint=True, ks=1.0, vs=1.0, scale=None,
        fused=False):
    kp, vp, table, k, v = make_cache(oracle, lens, h_kv, d, page, ks, vs, seed)
    g = torch.Generator().manual_seed(seed + 1)
    n = sum(new)
    wide = torch.randn((n + 4, h * d + (24 if fused else 0)), generator=g).to(dtype)
    wide[n:] = float("nan")
    q = (wide[:, 8:8 + h * d] if fused else wide).unflatten(1, (h, d))
    dev = wide.cuda()
    dev = (dev[:, 8:8 + h * d] if fused else dev).unflatten(1, (h, d))
    cq, ck = starts(new), starts(lens)
    out = torch.full((n + 4, h, d), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((h, n + 4), 7.0, device="cuda")
    args = (dev, kp.cuda(), vp.cuda(), table.cuda(), ints(cq), ints(lens))
    kw = dict(max_seqlen_q=max(new) if hint else 0, causal=causal, k_scale=ks, v_scale=vs, scale=scale)
    ea.attn_chunk_paged_q4(*args, out=out, lse=lse, **kw)
    assert ea.attn_get_device_status() == ea.ATTN_OK
    assert torch.all(out[n:] == 7.0) and torch.all(lse[:, n:] == 7.0)
    check(out, lse, q, k, v, cq, ck, causal, dtype, oracle, scale)
    again = ea.attn_chunk_paged_q4(*args, **kw)  # the same call, the same bits
    assert torch.equal(again[0][:n], out[:n]) and torch.equal(again[1][:, :n], lse[:, :n])


@pytest.mark.parametrize("page", [16, 48, 64, 256])
@pytest.mark.parametrize("hint", [False, True])
def test_one_token_each(gpu, oracle_mod, page, hint):
    lens = [1, 15, 16, 17, 128, 129, 1000, 2049, 0]
    run(gpu, oracle_mod, [1] * 9, lens, 8, 2, 128, page, torch.bfloat16, hint=hint)


@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("h,h_kv", [(4, 4), (6, 2), (5, 1), (16, 1), (24, 1), (64, 1)])
@pytest.mark.parametrize("new", [[1, 1, 1], [1, 7, 1], [2, 0, 1]])
def test_head_dims_and_groups(gpu, oracle_mod, d, dtype, h, h_kv, new):
    run(gpu, oracle_mod, new, [700, 300, 33], h, h_kv, d, 32, dtype, ks=0.37, vs=0.125, fused=d < 64)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("new,lens", [
    ([200, 1, 1, 64], [900, 1500, 3, 64]),     # chunks beside single tokens, a whole prompt
    ([0, 3, 0], [50, 40, 0]),                  # requests that bring nothing
    ([5, 2], [3, 0]),                          # rows before the first key, a request without keys
    ([4, 3, 1], [2, 130, 0]),
    ([300], [300]),
])
def test_chunks(gpu, oracle_mod, new, lens, causal):
    run(gpu, oracle_mod, new, lens, 8, 2, 128, 16, torch.bfloat16, causal)
    run(gpu, oracle_mod, new, lens, 3, 3, 64, 64, torch.float16, causal, ks=3.0, vs=0.5)
    run(gpu, oracle_mod, new, lens, 4, 2, 32, 48, torch.bfloat16, causal, hint=False)


@pytest.mark.parametrize("new", [1, 3, 6, 100])
def test_long_cache_is_cut(gpu, oracle_mod, new):
    run(gpu, oracle_mod, [new, 1], [20001, 130], 4, 1, 128, 64, torch.bfloat16)
    run(gpu, oracle_mod, [new, 1], [9000, 20], 2, 2, 32, 16, torch.float16)
    run(gpu, oracle_mod, [1, new], [70, 40007], 8, 1, 64, 16, torch.float16)


def test_many_requests(gpu, oracle_mod):
    r = np.random.default_rng(3)
    lens = [int(x) for x in r.integers(0, 200, 500)]
    run(gpu, oracle_mod, [1] * 500, lens, 4, 2, 64, 16, torch.bfloat16)
    run(gpu, oracle_mod, [int(x) for x in r.integers(0, 4, 500)], lens, 4, 2, 16, 16, torch.float16)


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("scale", [-0.3, 0.0, 1.7])
def test_scales(gpu, oracle_mod, new, scale):
    """A negative scale, none, and one under which the softmax sits on few keys."""
    run(gpu, oracle_mod, [new, 1], [600, 300], 4, 2, 64, 16, torch.bfloat16, scale=scale)
    run(gpu, oracle_mod, [new, 1], [600, 300], 4, 2, 128, 16, torch.float16, scale=scale, ks=2.0 ** -10, vs=2.0 ** 10)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("new", [1, 50])
def test_queries_of_very_different_sizes(gpu, oracle_mod, dtype, new):
    """Rows from 2^-12 to 2^12 (bf16: 2^-60 to 2^40 too), with values of every size in them and a row of zeros."""
    d, h, lens = 64, 4, [333]
    kp, vp, table, k, v = make_cache(oracle_mod, lens, 2, d, 16, 1.0, 1.0, 9)
    g = torch.Generator().manual_seed(2)
    q = torch.randn((new, h, d), generator=g)
    e = torch.tensor([-12.0, 12.0, 0.0, 3.0] if dtype == torch.float16 else [-60.0, 40.0, -12.0, 12.0])
    q = q * torch.exp2(e)[None, :, None] * torch.exp2(-12.0 * torch.rand(q.shape, generator=g))
    if new > 1:
        q[1] = 0.0
    q = q.to(dtype)
    cq, ck = starts([new]), starts(lens)
    for scale in (2.0 ** -6, 2.0 ** -40):
        o, lse = gpu.attn_chunk_paged_q4(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), ints(cq), ints(lens), new,
                                         scale=scale, causal=True)
        heads = range(h) if scale < 1e-6 or dtype == torch.float16 else (0, 2, 3)  # (2^34 as a score says nothing)
        for x in heads:
            check(o[:, x:x + 1], lse[x:x + 1], q[:, x:x + 1], k[:, x // 2:x // 2 + 1], v[:, x // 2:x // 2 + 1], cq, ck,
                  True, dtype, oracle_mod, scale)


def test_offsets_past_32_bits(gpu, oracle_mod):
    """Pools of more than 2^32 bytes: the pages at their end."""
    page, h_kv, d, h = 256, 8, 128, 16
    block = gpu.attn_q4_page_bytes(page, d)
    pool = (1 << 32) // (h_kv * block) + 9
    big = [torch.empty((pool, h_kv, block), dtype=torch.uint8, device="cuda") for _ in "kv"]
    lens = [700, 5]
    kp, vp, table, k, v = make_cache(oracle_mod, lens, h_kv, d, page, 1.0, 1.0, 11)
    for x, y in zip(big, (kp, vp)):
        x[pool - kp.shape[0]:] = y.cuda()
    table = torch.where((table >= 0) & (table < kp.shape[0]), table + pool - kp.shape[0], 0)
    g = torch.Generator().manual_seed(9)
    for new in ([2, 1], [40, 3]):
        q = torch.randn((sum(new), h, d), generator=g).to(torch.bfloat16)
        o, lse = gpu.attn_chunk_paged_q4(q.cuda(), *big, table.cuda(), ints(starts(new)), ints(lens), max(new),
                                         causal=True)
        assert gpu.attn_get_device_status() == gpu.ATTN_OK
        check(o, lse, q, k, v, starts(new), starts(lens), True, torch.bfloat16, oracle_mod)


def test_starts_and_lengths_that_make_no_sense(gpu, oracle_mod):
    """Lengths outside the table's are clamped; pages outside the pool too; starts out of order deal nothing out."""
    lens = [100, 60]
    kp, vp, table, k, v = make_cache(oracle_mod, lens, 2, 64, 16, 1.0, 1.0, 3)
    q = torch.randn((6, 4, 64), generator=torch.Generator().manual_seed(1)).to(torch.float16)
    for new in (1, 3):
        args = [q[:2 * new].cuda(), kp.cuda(), vp.cuda(), table.cuda(), ints([0, new, 2 * new])]
        want = gpu.attn_chunk_paged_q4(*args, ints([100, 0]), new, causal=True)
        got = gpu.attn_chunk_paged_q4(*args, ints([100, -5]), new, causal=True)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        gpu.attn_chunk_paged_q4(*args, ints([100, 1 << 30]), new, causal=True)
        out = torch.full_like(args[0], 7.0)
        gpu.attn_chunk_paged_q4(*args[:4], ints([0, 5 * new, new]), ints(lens), new, out=out, causal=True)
        assert gpu.attn_get_device_status() == gpu.ATTN_OK


def test_captured_and_on_two_streams(gpu, oracle_mod):
    lens, new = [5000, 700], [1, 3]
    kp, vp, table, k, v = make_cache(oracle_mod, lens, 2, 128, 16, 1.0, 1.0, 7)
    q = torch.randn((4, 8, 128), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    args = (q, kp.cuda(), vp.cuda(), table.cuda(), ints(starts(new)), ints(lens))
    for hint in (3, 0):
        want = gpu.attn_chunk_paged_q4(*args, hint, causal=True)
        outs = [torch.empty_like(x) for x in want], [torch.empty_like(x) for x in want]
        graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        torch.cuda.synchronize()
        for graph, (o, lse), side in zip(graphs, outs, streams):
            with torch.cuda.graph(graph, stream=side):
                for _ in range(3):
                    gpu.attn_chunk_paged_q4(*args, hint, out=o, lse=lse, causal=True)
        for _ in range(3):
            for o, lse in outs:
                o.zero_()
                lse.zero_()
            torch.cuda.synchronize()
            for graph, side in zip(graphs, streams):  # both at once
                with torch.cuda.stream(side):
                    graph.replay()
            torch.cuda.synchronize()
            for o, lse in outs:
                assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        many = [gpu.attn_chunk_paged_q4(*args, hint, causal=True, stream=s) for s in streams * 3]
        torch.cuda.synchronize()
        assert all(torch.equal(o, want[0]) and torch.equal(x, want[1]) for o, x in many)
        assert gpu.attn_get_device_status() == gpu.ATTN_OK


@pytest.mark.parametrize("h,h_kv,d,rot", [(8, 2, 128, 128), (4, 4, 64, 32), (16, 1, 64, 64)])
def test_serving_loop(gpu, oracle_mod, h, h_kv, d, rot):
    """Prompts, a step of single tokens, a mixed one: plan, append, attention,
    against attention over what attn_paged_read_q4 gives for the same rows."""
    page, b, far, dtype = 16, 3, 400, torch.bfloat16
    block = gpu.attn_q4_page_bytes(page, d)
    pools = [torch.full((60, h_kv, block), 0x7f, dtype=torch.uint8, device="cuda") for _ in "kv"]
    table = torch.full((b, 20), -1, dtype=torch.int32, device="cuda")
    free, count = ints(np.random.default_rng(2).permutation(60)), ints([60])
    lens = ints([0] * b)
    angle = np.arange(far)[:, None] * 100.0 ** (-np.arange(0, rot, 2) / rot)
    cs = torch.tensor(np.concatenate([np.cos(angle), np.sin(angle)], 1), dtype=torch.float32)
    g = torch.Generator().manual_seed(4)
    slots_of = [[] for _ in range(b)]
    keys = [0] * b
    for new in ([100, 33, 0], [1, 1, 1], [1, 60, 3], [1, 1, 1]):
        n = sum(new)
        q, k, v = (torch.randn((n, x, d), generator=g).to(dtype) for x in (h, h_kv, h_kv))
        pos = np.concatenate([np.arange(keys[i], keys[i] + m) for i, m in enumerate(new)])
        cu, lens, slots, count = gpu.attn_paged_plan(lens, ints(new), table, free, count, page, max_tokens=n)
        q_rot = gpu.attn_paged_append_q4(q.cuda(), k.cuda(), v.cuda(), cs.cuda(), ints(pos, torch.int64), slots, *pools,
                                         k_scale=0.5)
        o, lse = gpu.attn_chunk_paged_q4(q_rot, *pools, table, cu, lens, max(new), k_scale=0.5, causal=True)
        at = 0
        for i, m in enumerate(new):
            slots_of[i] += slots[at:at + m].tolist()
            keys[i] += m
            at += m
        where = np.concatenate(slots_of).astype(np.int64)
        kk, vv = gpu.attn_paged_read_q4(*pools, ints(where, torch.int64), d, k_scale=0.5)
        assert gpu.attn_get_device_status() == gpu.ATTN_OK
        check(o, lse, q_rot.cpu(), kk.double().cpu().numpy(), vv.double().cpu().numpy(), starts(new), starts(keys), True,
              dtype, oracle_mod)
        # and the keys are the rotated ones, within the format's steps: 1/6 of a group's largest, and the scale's
        ref = oracle_mod.rotate(k, cs, pos)
        mine = kk.double().cpu().numpy()[np.concatenate(
            [sum(keys[:i]) + keys[i] - m + np.arange(m) for i, m in enumerate(new)]).astype(int)]
        m = np.abs(ref.reshape(n, h_kv, -1, 16)).max(-1).repeat(16, -1).reshape(ref.shape)
        assert np.all(np.abs(mine - ref) <= m * (1 / 6 * 17 / 16 + 1 / 16 + 2.0 ** -8))
