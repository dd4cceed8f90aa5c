"""Chunks of new tokens over a paged cache (attn_chunk_paged), block tables and
slot maps (attn_paged_plan) and new rows into pages (attn_paged_write) against
the fp64 oracle, alone and as a serving loop runs them.
"""
import numpy as np
import pytest
import torch

from packed_parity import check_forward, default_scale, fp32_slack, starts

pytestmark = pytest.mark.gpu


def ints(x, dtype=torch.int32):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


def make_cache(lens, h_kv, d, page, dtype, seed, spare=3):
    """Shuffled pages whose rows past each request's end hold NaN, tables whose
    entries past it are out of range, and each request's keys in order."""
    g = torch.Generator().manual_seed(seed)
    n = [-(-m // page) for m in lens]
    width = max(max(n), 1) + 1
    pool = sum(n) + spare
    kp, vp = (torch.randn((pool, page, h_kv, d), generator=g).to(dtype) for _ in "kv")
    perm = torch.randperm(pool, generator=g).tolist()
    table = torch.tensor([[-1, 10 ** 6, pool][i % 3] for i in range(width)], dtype=torch.int32).repeat(len(lens), 1)
    keys, values = [], []
    for i, m in enumerate(lens):
        ids = [perm.pop() for _ in range(n[i])]
        table[i, :n[i]] = torch.tensor(ids, dtype=torch.int32)
        keys.append(kp[ids].flatten(0, 1)[:m].clone())
        values.append(vp[ids].flatten(0, 1)[:m].clone())
        if m % page:
            kp[ids[-1], m % page:] = float("nan")
            vp[ids[-1], m % page:] = float("nan")
    for i in perm:
        kp[i], vp[i] = float("nan"), float("inf")
    return kp, vp, table, torch.cat(keys), torch.cat(values)


def run(ea, oracle, new, lens, h, h_kv, d, page, dtype, causal=True, seed=5, hint=True):
    kp, vp, table, k, v = make_cache(lens, h_kv, d, page, dtype, seed)
    g = torch.Generator().manual_seed(seed + 1)
    n = sum(new)
    q = torch.randn((n + 4, h, d), generator=g).to(dtype)
    cq, ck, scale = starts(new), starts(lens), default_scale(d)
    out = torch.full((n + 4, h, d), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((h, n + 4), 7.0, device="cuda")
    ea.attn_chunk_paged(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), ints(cq), ints(lens),
                        max_seqlen_q=max(new) if hint else 0, out=out, lse=lse, causal=causal)
    assert ea.attn_get_device_status() == ea.ATTN_OK
    o_ref, l_ref = oracle.packed_attention(q, k, v, cq, ck, scale, causal)
    a_ref, _ = oracle.packed_attention(q, k, v.abs(), cq, ck, scale, causal)
    check_forward(out, lse, o_ref, l_ref, a_ref, dtype, fp32_slack(q, k, scale, d), n)
    assert torch.all(out[n:] == 7.0) and torch.all(lse[:, n:] == 7.0)


@pytest.mark.parametrize("page", [16, 48, 64, 256])
@pytest.mark.parametrize("hint", [False, True])
def test_one_token_each(gpu, oracle_mod, page, hint):
    lens = [1, 15, 16, 17, 128, 129, 1000, 2049, 0]
    run(gpu, oracle_mod, [1] * 9, lens, 8, 2, 128, page, torch.bfloat16, hint=hint)


@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("h,h_kv", [(4, 4), (6, 2), (5, 1), (64, 1)])
def test_head_dims_and_groups(gpu, oracle_mod, d, dtype, h, h_kv):
    run(gpu, oracle_mod, [1, 7, 1], [700, 300, 33], h, h_kv, d, 32, dtype)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("new,lens", [
    ([200, 1, 1, 64], [900, 1500, 3, 64]),     # chunks beside single tokens, a whole prompt
    ([0, 3, 0], [50, 40, 0]),                  # requests that bring nothing
    ([5, 2], [3, 0]),                          # rows before the first key, a request without keys
    ([300], [300]),
])
def test_chunks(gpu, oracle_mod, new, lens, causal):
    run(gpu, oracle_mod, new, lens, 8, 2, 128, 16, torch.bfloat16, causal)
    run(gpu, oracle_mod, new, lens, 3, 3, 64, 64, torch.float16, causal)


@pytest.mark.parametrize("new", [1, 6, 100])
def test_long_cache_is_cut(gpu, oracle_mod, new):
    run(gpu, oracle_mod, [new, 1], [20001, 130], 4, 1, 128, 64, torch.bfloat16)
    run(gpu, oracle_mod, [new, 1], [9000, 20], 2, 2, 32, 16, torch.float16)


def test_many_requests(gpu, oracle_mod):
    r = np.random.default_rng(3)
    lens = [int(x) for x in r.integers(0, 200, 500)]
    run(gpu, oracle_mod, [1] * 500, lens, 4, 2, 64, 16, torch.bfloat16)


def test_offsets_past_32_bits(gpu, oracle_mod):
    """A pool of more than 2^32 bytes (and 2^31 values) per tensor: the pages at its end."""
    page, h_kv, d = 256, 8, 128
    pool = (1 << 31) // (page * h_kv * d) + 9
    kp = torch.empty((pool, page, h_kv, d), dtype=torch.bfloat16, device="cuda")
    vp = torch.empty_like(kp)
    lens, new = [700, 5], [2, 1]
    g = torch.Generator().manual_seed(9)
    k, v = (torch.randn((705, h_kv, d), generator=g).to(torch.bfloat16) for _ in "kv")
    table = torch.tensor([[pool - 1, pool - 4, 0], [pool - 2, 0, 0]], dtype=torch.int32)
    slots = [int(table[i, j // page]) * page + j % page for i, m in enumerate(lens) for j in range(m)]
    gpu.attn_paged_write(k.cuda(), v.cuda(), ints(slots, torch.int64), kp, vp)
    q = torch.randn((3, 16, d), generator=g).to(torch.bfloat16)
    o, lse = gpu.attn_chunk_paged(q.cuda(), kp, vp, table.cuda(), ints(starts(new)), ints(lens), causal=True)
    assert gpu.attn_get_device_status() == gpu.ATTN_OK
    args = (starts(new), starts(lens), default_scale(d), True)
    o_ref, l_ref = oracle_mod.packed_attention(q, k, v, *args)
    a_ref, _ = oracle_mod.packed_attention(q, k, v.abs(), *args)
    check_forward(o, lse, o_ref, l_ref, a_ref, torch.bfloat16, fp32_slack(q, k, default_scale(d), d), 3)


# ---------------------------------------------------------------- tables and slots
def check_plan(ea, oracle, old, new, page, width, spare, seed, room=None, count=None):
    g = np.random.default_rng(seed)
    have = [min(-(-max(o, 0) // page), width) for o in old]
    ids = g.permutation(sum(have) + spare + 7)
    table = np.full((len(old), width), -1, dtype=np.int64)
    at = 0
    for i, n in enumerate(have):
        table[i, :n] = ids[at:at + n]
        at += n
    free = np.concatenate([ids[at:], [10 ** 6] * 3])
    count = spare if count is None else count
    room = sum(max(x, 0) for x in new) + 4 if room is None else room
    dev = [ints(x) for x in (old, new, table, free, [count])]
    before = [x.clone() for x in dev]
    cu, lens, slots, left = ea.attn_paged_plan(*dev, page, max_tokens=room)
    t2, cu2, lens2, slots2, left2 = oracle.paged_plan(old, new, table, free, count, page, room)
    for got, want in ((dev[2], t2), (cu, cu2), (lens, lens2), (slots, slots2), (left, [left2])):
        assert np.array_equal(got.cpu().numpy().astype(np.int64), np.asarray(want)), (got, want)
    for i in (0, 1, 3, 4):
        assert torch.equal(dev[i], before[i])
    # the inputs are as they were: the call can be repeated
    again = ea.attn_paged_plan(*dev, page, max_tokens=room)
    for x, y in zip(again, (cu, lens, slots, left)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("page", [1, 16, 48, 256])
@pytest.mark.parametrize("b", [1, 7, 300, 1024, 1025, 5000])
def test_plan(gpu, oracle_mod, page, b):
    r = np.random.default_rng(b + page)
    old = r.integers(0, 300, b)
    new = np.where(r.random(b) < 0.3, 0, r.integers(0, 60, b))
    need = int((-(-(old + new) // page) + old // -page).sum())
    check_plan(gpu, oracle_mod, old.tolist(), new.tolist(), page, int(-(-(old + new).max() // page)) + 1, need + 2, b)


def test_plan_edges(gpu, oracle_mod):
    check_plan(gpu, oracle_mod, [0], [1], 16, 4, 1, 1)
    check_plan(gpu, oracle_mod, [0, 0, 0], [0, 0, 0], 16, 4, 1, 2)
    check_plan(gpu, oracle_mod, [16, 15, 17], [1, 1, 15], 16, 4, 9, 3)             # a page's first and last row
    check_plan(gpu, oracle_mod, [60, 3], [30, 2], 16, 4, 9, 4)                     # past the table's width
    check_plan(gpu, oracle_mod, [100, 3], [30, 2], 16, 4, 9, 4)                    # past it already
    check_plan(gpu, oracle_mod, [0, 0, 5], [40, 40, 40], 16, 4, 4, 5)              # pages run out
    check_plan(gpu, oracle_mod, [0, 0], [40, 40], 16, 4, 0, 6)                     # none at all
    check_plan(gpu, oracle_mod, [5, 6], [40, 40], 16, 4, 9, 7, room=50)            # a slot map that is too short
    check_plan(gpu, oracle_mod, [5, 6], [4, 4], 16, 4, 9, 8, room=5000)            # and one with much room
    check_plan(gpu, oracle_mod, [-3, 6], [4, -9], 16, 4, 9, 9)                     # negative lengths count as 0
    check_plan(gpu, oracle_mod, [5, 6], [40, 40], 16, 4, 9, 10, count=-4)          # a count out of range
    check_plan(gpu, oracle_mod, [0], [100000], 64, 2000, 1900, 11)                 # one long prompt


@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("h_kv", [1, 3, 8])
@pytest.mark.parametrize("tokens", [1, 5, 1000])
@pytest.mark.parametrize("fused", [False, True])
def test_write(gpu, d, h_kv, tokens, fused):
    page = 16
    pool = -(-tokens // page) + 2
    kp, vp = (torch.randn((pool, page, h_kv, d), device="cuda").half() for _ in "kv")
    slots = torch.randperm(pool * page)[:tokens]
    if tokens > 3:
        slots[1], slots[2], slots[3] = -1, pool * page, 2 ** 40
    wide = torch.randn((tokens, 2 * h_kv * d + 8), device="cuda").half()
    k, v = wide[:, 8:8 + h_kv * d].unflatten(1, (h_kv, d)), wide[:, 8 + h_kv * d:].unflatten(1, (h_kv, d))
    if not fused:
        k, v = k.contiguous(), v.contiguous()
    want = [kp.clone().flatten(0, 1), vp.clone().flatten(0, 1)]
    keep = ((slots >= 0) & (slots < pool * page)).nonzero()[:, 0]
    for x, y in zip(want, (k, v)):
        x[slots[keep].cuda()] = y[keep.cuda()]
    gpu.attn_paged_write(k, v, slots.cuda(), kp, vp)
    assert torch.equal(kp.flatten(0, 1), want[0]) and torch.equal(vp.flatten(0, 1), want[1])


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("graph", [False, True])
def test_serving_loop(gpu, oracle_mod, graph):
    """Prompts in chunks, then decoding, for requests that come at different
    times: plan, write, attend, each step checked; captured once and replayed
    with other lengths where ``graph``."""
    h, h_kv, d, page, width, b = 8, 2, 64, 16, 12, 4
    dtype, scale, room = torch.bfloat16, default_scale(64), 70
    g = torch.Generator().manual_seed(31)
    steps = [[30, 0, 1, 0], [40, 17, 1, 0], [1, 1, 1, 50], [1, 1, 1, 1], [0, 30, 1, 1], [1, 1, 1, 1]]
    pool = b * width
    kp, vp = (torch.full((pool, page, h_kv, d), float("nan"), dtype=dtype, device="cuda") for _ in "kv")
    table = torch.full((b, width), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(pool, generator=g).to(torch.int32).cuda()
    count, lens = ints([pool]), ints([0] * b)
    new = ints([0] * b)
    q, k, v = (torch.zeros((room, n, d), dtype=dtype, device="cuda") for n in (h, h_kv, h_kv))
    out, lse = torch.empty((room, h, d), dtype=dtype, device="cuda"), torch.empty((h, room), device="cuda")
    cu, lens2, left = ints([0] * (b + 1)), ints([0] * b), ints([0])
    slots = torch.empty(room, dtype=torch.int64, device="cuda")

    def step():
        gpu.attn_paged_plan(lens, new, table, free, count, page, cu_seqlens_q=cu, seqlens_out=lens2,
                            slot_map=slots, free_left=left)
        gpu.attn_paged_write(k, v, slots, kp, vp)
        gpu.attn_chunk_paged(q, kp, vp, table, cu, lens2, out=out, lse=lse, causal=True)
        lens.copy_(lens2)
        count.copy_(left)

    run_step = step
    if graph:
        step()  # with no token at all
        torch.cuda.synchronize()
        recorded = torch.cuda.CUDAGraph()
        with torch.cuda.graph(recorded):
            step()
        run_step = recorded.replay
    past = [[torch.zeros((0, h_kv, d), dtype=dtype)] * 2 for _ in range(b)]
    for fresh in steps:
        n = sum(fresh)
        rows = [torch.randn((n, x, d), generator=g).to(dtype) for x in (h, h_kv, h_kv)]
        for x, y in zip((q, k, v), rows):
            x[:n] = y.cuda()
        new.copy_(ints(fresh))
        run_step()
        assert gpu.attn_get_device_status() == gpu.ATTN_OK
        cq = starts(fresh)
        for i in range(b):
            past[i] = [torch.cat([old, y[cq[i]:cq[i + 1]]]) for old, y in zip(past[i], rows[1:])]
        keys, values = (torch.cat([x[j] for x in past]) for j in (0, 1))
        ck = starts([x[0].shape[0] for x in past])
        assert lens.tolist() == np.diff(ck).tolist()
        o_ref, l_ref = oracle_mod.packed_attention(rows[0], keys, values, cq, ck, scale, True)
        a_ref, _ = oracle_mod.packed_attention(rows[0], keys, values.abs(), cq, ck, scale, True)
        check_forward(out, lse, o_ref, l_ref, a_ref, dtype, fp32_slack(rows[0], keys, scale, d), n)
    used = sum(-(-n // page) for n in lens.tolist())
    assert count.item() == pool - used


def test_skipped_loads_time_out_and_recover(gpu):
    kp, vp, table, _, _ = make_cache([300], 2, 128, 16, torch.bfloat16, 3)
    args = [torch.randn(1, 4, 128).bfloat16().cuda(), kp.cuda(), vp.cuda(), table.cuda(), ints([0, 1]), ints([300])]
    first, _ = gpu.attn_chunk_paged(*args)
    gpu.attn_debug_set_flags(gpu.ATTN_DEBUG_SKIP_LOADS)
    try:
        gpu.attn_chunk_paged(*args)
    finally:
        gpu.attn_debug_set_flags(0)
    assert gpu.attn_get_device_status() == gpu.ATTN_ERR_DEVICE_TIMEOUT
    again, _ = gpu.attn_chunk_paged(*args)
    assert gpu.attn_get_device_status() == gpu.ATTN_OK
    assert torch.equal(first, again)
