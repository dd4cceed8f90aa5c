"""Rotation and rows into pages (attn_paged_append, attn_paged_append_q4) and
rows out of a 4-bit cache (attn_paged_read_q4) against float64.

Bounds, with u = eps / 2 of the 16-bit type and f = 2^-24: a rotated value has
two rounded products and a rounded sum, |a c| + |b s| times 2 f at most (the
table is taken as it is), and is rounded once: 2 f (|a| + |b|) + u max(|x|, the
least normal number). A
4-bit row's scale is the oracle's of an m moved by that much, and its code is as
near as the best one but for the same error (and as much again for the
quotient): bits are equal where nothing turns.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
F = 2.0 ** -24
NAN = float("nan")


def ints(x, dtype=torch.int64):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


def table(far, rot):
    angle = np.arange(far)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
    return torch.tensor(np.concatenate([np.cos(angle), np.sin(angle)], 1), dtype=torch.float32)


def rows(t, heads, d, dtype, g, fused):
    wide = torch.randn((t, heads * d + (24 if fused else 0)), generator=g).to(dtype)
    x = wide.cuda()
    x = x[:, 8:8 + heads * d] if fused else x
    return x.unflatten(1, (heads, d))


def step(t, h, h_kv, d, rot, dtype, seed, fused=False, far=500):
    g = torch.Generator().manual_seed(seed)
    q, k, v = (rows(t, n, d, dtype, g, fused) for n in (h, h_kv, h_kv))
    r = np.random.default_rng(seed)
    pos = r.integers(0, far, t)
    pos[0] = far - 1
    return q, k, v, table(far, rot), pos


def turned(oracle, x, cs, pos, interleaved):
    """The rotated rows in float64, and |a| + |b| of each value's pair."""
    ref = oracle.rotate(x.cpu(), cs, pos, interleaved)
    a, rot = np.abs(x.double().cpu().numpy()), cs.shape[1]
    size = np.zeros_like(a)
    if interleaved:
        size[..., :rot] = np.repeat(a[..., 0:rot:2] + a[..., 1:rot:2], 2, -1)
    else:
        size[..., :rot] = np.tile(a[..., :rot // 2] + a[..., rot // 2:rot], 2)
    return ref, size


def check_turned(got, ref, size, dtype):
    u = torch.finfo(dtype).eps / 2
    err = np.abs(got.double().cpu().numpy() - ref)
    over = err - (u * np.maximum(np.abs(ref), torch.finfo(dtype).tiny) + (1 + u) * 2 * F * size)
    assert over.max() <= 0, f"off by {err.max():.3e}, {over.max():.3e} over its bound"
    assert np.all(err[size == 0] == 0)


SHAPES = [  # t, h, h_kv, d, rot, page, interleaved
    (1, 32, 8, 128, 128, 16, False), (1, 4, 4, 16, 16, 16, True), (37, 32, 8, 128, 64, 48, False),
    (37, 5, 1, 64, 64, 16, True), (200, 16, 16, 64, 48, 64, False), (3, 1, 1, 32, 16, 256, False),
    (1000, 3, 3, 16, 16, 32, False), (129, 7, 5, 128, 112, 16, True), (63, 100, 2, 32, 32, 16, False),
]


@pytest.mark.parametrize("t,h,h_kv,d,rot,page,interleaved", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("fused", [False, True])
def test_append(gpu, oracle_mod, t, h, h_kv, d, rot, page, interleaved, dtype, fused):
    q, k, v, cs, pos = step(t, h, h_kv, d, rot, dtype, t + d, fused)
    pages = t // page + 3
    r = np.random.default_rng(t)
    slots = r.permutation(pages * page)[:t]
    if t > 4:
        slots[[2, t - 1]] = -1, pages * page  # padding tokens
    kp, vp = (torch.full((pages, page, h_kv, d), 7.0, dtype=dtype, device="cuda") for _ in "kv")
    out = torch.full((t + 2, h, d), 7.0, dtype=dtype, device="cuda")
    got = gpu.attn_paged_append(q, k, v, cs.cuda(), ints(pos), ints(slots), kp, vp, q_out=out[1:t + 1],
                                interleaved=interleaved)
    assert gpu.attn_get_device_status() == gpu.ATTN_OK
    assert got.data_ptr() == out[1:].data_ptr() and torch.all(out[0] == 7) and torch.all(out[t + 1] == 7)
    check_turned(got, *turned(oracle_mod, q, cs, pos, interleaved), dtype)
    keep = (slots >= 0) & (slots < pages * page)
    flat_k, flat_v = kp.flatten(0, 1), vp.flatten(0, 1)
    ref, size = turned(oracle_mod, k, cs, pos, interleaved)
    check_turned(flat_k[ints(slots[keep])], ref[keep], size[keep], dtype)
    assert torch.equal(flat_v[ints(slots[keep])], v[ints(np.flatnonzero(keep))])
    rest = np.setdiff1d(np.arange(pages * page), slots)
    assert torch.all(flat_k[ints(rest)] == 7) and torch.all(flat_v[ints(rest)] == 7)


def check_q4(oracle, pool, slots, ref, size, d, scale):
    """Rows of a 4-bit pool against float64 rows known up to 2 f size."""
    code, s = (x[slots] for x in oracle.q4_rows(pool.cpu().numpy(), d))
    slack = 2 * F * size
    group = lambda x: x.reshape(*x.shape[:-1], -1, 16)  # noqa: E731
    m = np.abs(group(ref))
    # (a quotient by a power of two is exact, another one rounded)
    exact = (group(size).max(-1) == 0) & (np.frexp(scale)[0] == 0.5)
    lo, hi = (oracle.nearest(oracle.E4M3, np.where(exact, m.max(-1), np.maximum(
        (m + sign * group(slack)).max(-1) * (1 + sign * 3 * F), 0)) / (6.0 * scale)) for sign in (-1, 1))
    assert np.all((s >= lo) & (s <= hi)), "a group's scale"
    unit = np.repeat(oracle.E4M3[s] * scale, 16, -1)
    y = np.where(unit > 0, ref / np.where(unit > 0, unit, 1.0), 0.0)
    best = np.abs(np.minimum(np.abs(y), 6.0) - oracle.E2M1[oracle.nearest(oracle.E2M1, y)])
    value = oracle.E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
    err = np.abs(np.clip(y, -6.0, 6.0) - value)
    wide = np.where(unit > 0, slack / np.where(unit > 0, unit, 1.0), 0.0)
    assert np.all(err <= best + 2 * (wide + 4 * F * np.abs(y))), "a code that is not the nearest"


@pytest.mark.parametrize("t,h,h_kv,d,rot,page,interleaved", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("fused,ks,vs", [(False, 1.0, 1.0), (True, 0.37, 0.125)])
def test_append_q4_and_read(gpu, oracle_mod, t, h, h_kv, d, rot, page, interleaved, dtype, fused, ks, vs):
    q, k, v, cs, pos = step(t, h, h_kv, d, rot, dtype, t + d + 1, fused)
    pages = t // page + 3
    slots = np.random.default_rng(t).permutation(pages * page)[:t]
    if t > 4:
        slots[[2, t - 1]] = -1, pages * page
    keep = (slots >= 0) & (slots < pages * page)
    kp, vp = (torch.full((pages, h_kv, gpu.attn_q4_page_bytes(page, d)), 0x5A, dtype=torch.uint8, device="cuda")
              for _ in "kv")
    got = gpu.attn_paged_append_q4(q, k, v, cs.cuda(), ints(pos), ints(slots), kp, vp, k_scale=ks, v_scale=vs,
                                   interleaved=interleaved)
    assert gpu.attn_get_device_status() == gpu.ATTN_OK
    check_turned(got, *turned(oracle_mod, q, cs, pos, interleaved), dtype)
    ref, size = turned(oracle_mod, k, cs, pos, interleaved)
    check_q4(oracle_mod, kp, slots[keep], ref[keep], size[keep], d, float(np.float32(ks)))
    # v does not turn: with a power of two as its scale the bits are the oracle's, ties included
    code, s = oracle_mod.q4_rows(vp.cpu().numpy(), d)
    want = oracle_mod.q4_quantise(v.cpu()[np.flatnonzero(keep)], vs)
    assert np.array_equal(s[slots[keep]], want[1])
    same = code[slots[keep]] == want[0]
    assert np.all(same | ((code[slots[keep]] | want[0]) == 8)), "codes (0 has two)"
    for pool in (kp, vp):
        rest = np.setdiff1d(np.arange(pages * page), slots)
        code, s = oracle_mod.q4_rows(pool.cpu().numpy(), d)
        assert np.all(s[rest] == 0x5A) and np.all(code[rest][..., 0::2] == 0xA) and np.all(code[rest][..., 1::2] == 5)
    # and back: the value, rounded once
    wide = torch.full((t, h_kv * d + 16), 7.0, dtype=dtype, device="cuda")
    k2, v2 = gpu.attn_paged_read_q4(kp, vp, ints(slots), d, k_scale=ks, v_scale=vs,
                                    k=wide[:, 8:8 + h_kv * d].unflatten(1, (h_kv, d)))
    assert torch.all(wide[:, :8] == 7) and torch.all(wide[:, 8 + h_kv * d:] == 7) and v2.dtype == dtype
    for x, pool, scale in ((k2, kp, ks), (v2, vp, vs)):
        value = oracle_mod.q4_values(*(y[slots[keep]] for y in oracle_mod.q4_rows(pool.cpu().numpy(), d)),
                                     float(np.float32(scale)))
        err = np.abs(x[ints(np.flatnonzero(keep))].double().cpu().numpy() - value)
        # (products with a scale that is no power of two are rounded in fp32; below
        # the type's normal numbers steps have one size)
        info = torch.finfo(dtype)
        assert np.all(err <= np.maximum((info.eps / 2 + 2 * F) * np.abs(value), info.tiny * info.eps / 2))
        assert torch.all(x[ints(np.flatnonzero(~keep))] == 0)


def test_positions_outside_the_table(gpu):
    """Nothing is written for such a token, wherever its slot is."""
    q, k, v, cs, pos = step(6, 4, 2, 64, 64, torch.bfloat16, 3)
    pos[[1, 3]] = -1, 500
    pos[4] = 1 << 40
    out = torch.full_like(q, 7.0)
    kp, vp = (torch.full((1, 16, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    gpu.attn_paged_append(q, k, v, cs.cuda(), ints(pos), ints(range(6)), kp, vp, q_out=out)
    for x in (out, kp[0, :6], vp[0, :6]):
        untouched = [bool(torch.all(x[i] == 7)) for i in range(6)]
        assert untouched == [False, True, False, True, True, False]
    k4, v4 = (torch.full((1, 2, gpu.attn_q4_page_bytes(16, 64)), 0x33, dtype=torch.uint8, device="cuda") for _ in "kv")
    out.fill_(7.0)
    gpu.attn_paged_append_q4(q, k, v, cs.cuda(), ints(pos), ints(range(6)), k4, v4, q_out=out)
    codes = v4[0, :, :16 * 32].unflatten(1, (16, 32))
    assert [bool(torch.all(codes[:, i] == 0x33)) for i in range(6)] == [False, True, False, True, True, False]
    assert [bool(torch.all(out[i] == 7)) for i in range(6)] == [False, True, False, True, True, False]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(128, 128), (64, 32), (16, 16)])
def test_queries_in_place(gpu, d, rot, interleaved):
    q, k, v, cs, pos = step(50, 9, 3, d, rot, torch.float16, 8, fused=True)
    pages = [torch.zeros((5, 16, 3, d), dtype=torch.float16, device="cuda") for _ in range(4)]
    args = (k, v, cs.cuda(), ints(pos), ints(range(50)))
    want = gpu.attn_paged_append(q, *args, *pages[:2], interleaved=interleaved)
    got = gpu.attn_paged_append(q, *args, *pages[2:], q_out=q, interleaved=interleaved)
    assert got.data_ptr() == q.data_ptr() and torch.equal(got, want)
    assert torch.equal(pages[0], pages[2]) and torch.equal(pages[1], pages[3])


def test_values_that_a_scale_cannot_hold(gpu, oracle_mod):
    """Groups of zeros, below the least scale, above the largest, with an infinity or a NaN; borders of codes."""
    d = 16
    unit = 1.5  # 1.5 and 1.25 are e4m3 values
    borders = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0]
    x = torch.zeros((10, 1, d))
    x[1, 0] = 2.0 ** -11                                  # m / 6 rounds to a scale of 0
    x[2, 0, :3] = torch.tensor([60000.0, -3000.0, 100.0])  # more than 6 * 448
    x[3, 0, 5] = float("inf")
    x[4, 0, 5] = NAN
    x[5, 0, :16] = torch.tensor([s * b * unit for b in borders for s in (1, -1)])
    x[6, 0, :16] = torch.tensor([s * b * 1.25 for b in borders for s in (1, -1)])
    x[7, 0, 0] = 6 * (1 + 1 / 16)                          # a border between two scales: 1
    x[8, 0, 0] = 6 * (1 + 3 / 16)                          # and one up: 1.25
    x[9, 0, 15] = -float("inf")
    for dtype in (torch.float16, torch.bfloat16):
        v = x.to(dtype).cuda()
        q = torch.zeros_like(v)
        cs = table(4, 16).cuda()
        kp, vp = (torch.zeros((1, 1, gpu.attn_q4_page_bytes(16, d)), dtype=torch.uint8, device="cuda") for _ in "kv")
        gpu.attn_paged_append_q4(q, v, v, cs, ints([0] * 10), ints(range(10)), kp, vp)
        for pool in (kp, vp):  # (position 0 turns nothing: cos 1, sin 0; but an infinity there gives a NaN)
            code, s = (y[:10] for y in oracle_mod.q4_rows(pool.cpu().numpy(), d))
            want, ws = oracle_mod.q4_quantise(v.cpu(), 1.0)
            assert np.array_equal(s, ws)
            fine = ws[:, 0, 0] != 127
            assert fine.tolist() == [True] * 3 + [False] * 2 + [True] * 4 + [False]
            assert np.all((code[fine] == want[fine]) | ((code[fine] | want[fine]) == 8))
        back, _ = gpu.attn_paged_read_q4(kp, vp, ints(range(10)), d, dtype=dtype)
        assert torch.all(torch.isnan(back[3:5])) and torch.all(torch.isnan(back[9])) and torch.all(back[:2] == 0)


def test_offsets_past_32_bits(gpu, oracle_mod):
    """Pools of more than 2^32 bytes: their last pages."""
    page, h_kv, d, t = 64, 8, 128, 40
    q, k, v, cs, pos = step(t, 8, h_kv, d, d, torch.bfloat16, 4)
    block = gpu.attn_q4_page_bytes(page, d)
    pages = (1 << 32) // (h_kv * block) + 5
    kp, vp = (torch.empty((pages, h_kv, block), dtype=torch.uint8, device="cuda") for _ in "kv")
    slots = pages * page - 1 - np.arange(t)
    gpu.attn_paged_append_q4(q, k, v, cs.cuda(), ints(pos), ints(slots), kp, vp)
    last = vp[-1:].cpu().numpy()
    code, s = (x[page - 1 - np.arange(t)] for x in oracle_mod.q4_rows(last, d))
    want = oracle_mod.q4_quantise(v.cpu(), 1.0)
    assert np.array_equal(s, want[1]) and np.all((code == want[0]) | ((code | want[0]) == 8))
    _, back = gpu.attn_paged_read_q4(kp, vp, ints(slots), d)
    assert np.array_equal(back.double().cpu().numpy(), oracle_mod.q4_values(*want, 1.0))
    pages = (1 << 31) // (page * h_kv * d) + 3
    kp, vp = (torch.empty((pages, page, h_kv, d), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    slots = pages * page - 1 - np.arange(t)
    gpu.attn_paged_append(q, k, v, cs.cuda(), ints(pos), ints(slots), kp, vp)
    assert torch.equal(vp[-1][ints(page - 1 - np.arange(t))], v)


def test_captured_and_on_another_stream(gpu):
    q, k, v, cs, pos = step(70, 8, 2, 64, 64, torch.bfloat16, 12)
    pools = [torch.zeros((6, 2, gpu.attn_q4_page_bytes(16, 64)), dtype=torch.uint8, device="cuda") for _ in range(4)]
    args = (q, k, v, cs.cuda(), ints(pos), ints(range(70)))
    want_q = gpu.attn_paged_append_q4(*args, *pools[:2])
    want = gpu.attn_paged_read_q4(*pools[:2], args[5], 64)
    side = torch.cuda.Stream()
    out = torch.empty_like(q)
    got = [torch.empty_like(x) for x in want]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        gpu.attn_paged_append_q4(*args, *pools[2:], q_out=out)
        gpu.attn_paged_read_q4(*pools[2:], args[5], 64, k=got[0], v=got[1])
    for _ in range(2):
        out.zero_()
        for x in pools[2:]:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want_q) and all(torch.equal(a, b) for a, b in zip(got, want))
    for x in pools[2:]:
        x.zero_()
    torch.cuda.synchronize()
    made = gpu.attn_paged_append_q4(*args, *pools[2:], stream=side)
    side.synchronize()
    assert torch.equal(made, want_q) and torch.equal(pools[2], pools[0]) and torch.equal(pools[3], pools[1])
