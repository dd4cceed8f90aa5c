"""Starts of packed sequences as the kernels read them from the device, whatever
they hold, on the host: rows stay inside the tensors, and starts out of order,
whose sequences could overlap and make the 32-bit sums of the work line wrap,
deal nothing out.
"""
import ctypes
import random

import pytest
import torch

import exact_attention_65_gb300 as ea
from test_packed_abi import BWD, BWD_OK, CHUNK, CHUNK_OK, FWD, FWD_OK, call
from test_packed_plan import FIELDS, plan


def deal(lib, cq, ck, total_q, total_k, h, h_kv, one_tile, causal, by_key, ctas=152):
    b = len(cq) - 1
    room = 1 << 20
    out = (ctypes.c_int * (9 * room))()
    q, k = ((ctypes.c_int * (b + 1))(*x) for x in (cq, ck))
    n = lib.attn_debug_packed_starts(q, k, b, total_q, total_k, h, h_kv, one_tile, causal, by_key, ctas, room, out)
    assert 0 <= n < room
    return [dict(zip(FIELDS, out[9 * i:9 * i + 9])) for i in range(n)]


@pytest.mark.parametrize("by_key", [0, 1])
@pytest.mark.parametrize("one_tile", [0, 1])
@pytest.mark.parametrize("b,rows", [(64, 1 << 20), (6000, 1 << 16), (2, 5), (33, 64)])
def test_overlapping_sequences_deal_nothing(exattn_lib, b, rows, one_tile, by_key):
    """Starts that alternate between 0 and the end: every other sequence has all
    rows. 64 of 2^20 rows cost more than 2^31 together."""
    cu = [0 if i % 2 == 0 else rows for i in range(b + 1)]
    assert deal(exattn_lib, cu, cu, rows, rows, 32, 8, one_tile, 1, by_key) == []


@pytest.mark.parametrize("by_key", [0, 1])
@pytest.mark.parametrize("b", [1, 5, 32, 33, 70])
def test_one_start_out_of_order_anywhere(exattn_lib, b, by_key):
    """In either array, at every place: nothing; put right, everything."""
    good = [10 * i for i in range(b + 1)]
    assert deal(exattn_lib, good, good, 10 * b, 10 * b, 4, 2, 0, 1, by_key)
    for at in sorted({0, b // 2, b - 1}):
        bad = list(good)
        bad[at] = bad[at + 1] + 1
        assert deal(exattn_lib, bad, good, 10 * b, 10 * b, 4, 2, 0, 1, by_key) == []
        assert deal(exattn_lib, good, bad, 10 * b, 10 * b, 4, 2, 0, 1, by_key) == []


def test_rows_stay_inside_the_tensors(exattn_lib):
    """Starts in order but past the ends are the same as clamped ones."""
    r = random.Random(7)
    for _ in range(60):
        b, total = r.choice([1, 3, 40]), r.choice([1, 64, 3000])
        cq, ck = (sorted(r.choice([-2 ** 31, -5, 0, total, 2 ** 31 - 1, r.randint(0, total)]) for _ in range(b + 1))
                  for _ in "qk")
        cut = [[min(max(x, 0), total) for x in c] for c in (cq, ck)]
        sq, sk = ([z - a for a, z in zip(c, c[1:])] for c in cut)
        args = (4, 1, r.randrange(2), r.randrange(2), r.randrange(2))
        got = deal(exattn_lib, cq, ck, total, total, *args)
        assert got == deal(exattn_lib, *cut, total, total, *args)
        units = {(x["seq"], x["unit"]) for x in got}
        length = 128 if args[4] else 32 * (1 if args[2] else 2)
        for seq, unit in units:
            assert unit * length < (sk if args[4] else sq)[seq]


def test_the_first_part_of_a_cut_unit_is_never_before_the_line(exattn_lib):
    for sq, sk in (([1], [32768]), ([5000, 3, 9000], [5000, 700, 9000]), ([1] * 40, [3000] * 40)):
        for by_key in (0, 1):
            for r in plan(exattn_lib, sq, sk, 32, 8, 1, 1, by_key):
                assert 0 <= r["first"] <= r["cta"] < r["first"] + r["nparts"]


@pytest.mark.parametrize("fn,order,ok,kw", [
    ("attn_fwd_packed", FWD, FWD_OK, dict(tq=65535)),
    ("attn_bwd_packed", BWD, BWD_OK, dict(tq=65535)),
    ("attn_bwd_packed", BWD, BWD_OK, dict(tq=1, tk=65535)),
    ("attn_chunk_paged", CHUNK, CHUNK_OK, dict(tq=65535)),
])
def test_refuses_more_units_than_are_counted(exattn_lib, fn, order, ok, kw):
    """65,535 requests of a row each times 65,535 heads."""
    wide = {x: 65535 * 16 for x in ("qs", "ks", "vs", "dqs", "dks", "dvs")}
    args = dict(ok, b=65535, h=65535, hk=65535, d=16, **wide, **kw)
    assert call(getattr(exattn_lib, fn), order, **args) == ea.ATTN_ERR_UNSUPPORTED


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def guarded(rows, *tail, dtype=torch.float16):
    """Room for `rows` rows between two rows of 7.0."""
    x = torch.full((rows + 2, *tail), 7.0, dtype=dtype, device="cuda")
    return x, x[1:rows + 1]


def untouched(x):
    return bool(torch.all(x[0] == 7.0) and torch.all(x[-1] == 7.0))


OUT_OF_ORDER = [
    (64, [0, 64, 0, 64]),
    (64, [64, 10, 64, 64]),
    (300, [0] + [300, 0] * 35 + [300]),                    # more than 32 sequences
    (1 << 20, [(1 << 20) * (i % 2) for i in range(65)]),   # costs that wrap
]


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cu", OUT_OF_ORDER, ids=["three", "descending", "many", "wrapping"])
@pytest.mark.parametrize("hint", [0, 1])
def test_nothing_outside_the_tensors_is_touched(gpu, rows, cu, hint):
    h, h_kv, d = 4, 1, 16
    q, k, v = (torch.randn(rows, n, d, device="cuda").half() for n in (h, h_kv, h_kv))
    starts = ints(cu)
    frame, out = guarded(rows, h, d)
    lse_frame = torch.full((h * rows + 2,), 7.0, device="cuda")
    lse = lse_frame[1:-1].view(h, rows)
    gpu.attn_fwd_packed(q, k, v, starts, starts, max_seqlen_q=hint, out=out, lse=lse, causal=True)
    frames = [guarded(rows, n, d) for n in (h, h_kv, h_kv)]
    gpu.attn_bwd_packed(q, k, v, torch.zeros_like(q), torch.zeros(h, rows, device="cuda"), torch.randn_like(q), starts,
                        starts, dq=frames[0][1], dk=frames[1][1], dv=frames[2][1], causal=True)
    b = len(cu) - 1
    pages = torch.randn(8, 16, h_kv, d, device="cuda").half()
    table = torch.zeros(b, 2, dtype=torch.int32, device="cuda")
    paged_frame, paged = guarded(rows, h, d)
    gpu.attn_chunk_paged(q, pages, pages.clone(), table, starts, ints([20] * b), max_seqlen_q=hint, out=paged, causal=True)
    assert gpu.attn_get_device_status() == gpu.ATTN_OK
    assert all(untouched(x) for x in (frame, paged_frame, *(x for x, _ in frames)))
    assert lse_frame[0] == 7.0 and lse_frame[-1] == 7.0
    # and the next call is as ever
    good = ints([0, rows // 2, rows])
    first = gpu.attn_fwd_packed(q, k, v, good, good, causal=True)
    again = gpu.attn_fwd_packed(q, k, v, good, good, causal=True)
    assert all(torch.equal(x, y) for x, y in zip(first, again)) and torch.isfinite(first[0].float()).all()
