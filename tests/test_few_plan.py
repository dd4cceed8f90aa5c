"""How requests with few rows over a 4-bit cache are dealt to warps, on the host
(the kernel runs the same arithmetic): every unit's steps of 32 keys are covered
exactly once, in order; the warps that share a cut unit are neighbours and agree
on who they are, each with a step at least; no warp gets much more than its
share.
"""
import ctypes
import random

import pytest

FIELDS = ("warp", "seq", "head", "unit", "step0", "nstep", "slot", "first", "nparts")


def plan(lib, sq, sk, h, h_kv, rows, causal, warps):
    b, room = len(sq), 1 << 17
    out = (ctypes.c_int * (9 * room))()
    n = lib.attn_debug_few_plan((ctypes.c_int * b)(*sq), (ctypes.c_int * b)(*sk), b, h, h_kv, rows, causal, warps, room,
                                out)
    assert 0 <= n < room
    return [dict(zip(FIELDS, out[9 * i:9 * i + 9])) for i in range(n)]


def check(lib, sq, sk, h, h_kv, rows, causal, warps):
    tokens = rows // (h // h_kv)
    ranges = plan(lib, sq, sk, h, h_kv, rows, causal, warps)
    want = {}
    for s, (n, m) in enumerate(zip(sq, sk)):
        for head in range(h_kv):
            for unit in range(-(-n // tokens)):
                last = min((unit + 1) * tokens, n) - 1
                keys = max(0, min(m, last + m - n + 1)) if causal else m
                want[s, head, unit] = -(-keys // 32)
    at, shares, work = {}, {}, {}
    for r in ranges:
        key = r["seq"], r["head"], r["unit"]
        assert r["step0"] == at.get(key, 0), "a gap or an overlap"
        at[key] = r["step0"] + r["nstep"]
        assert r["nstep"] > 0 or want[key] == 0
        assert (r["slot"] < 0) == (r["nstep"] == want[key])
        if r["slot"] >= 0:
            assert r["slot"] == (0 if r["step0"] > 0 else 1)
            shares.setdefault(key, []).append(r)
        work[r["warp"]] = work.get(r["warp"], 0) + r["nstep"] + 2
    assert at == want
    assert [r["warp"] for r in ranges] == sorted(r["warp"] for r in ranges)
    for parts in shares.values():
        assert [r["warp"] for r in parts] == list(range(parts[0]["warp"], parts[0]["warp"] + len(parts)))
        assert all(r["first"] == parts[0]["warp"] and r["nparts"] == len(parts) for r in parts)
        # a warp whose share ends inside the unit has nothing behind it
        for r in parts[:-1]:
            assert max(i for i, x in enumerate(ranges) if x["warp"] == r["warp"]) == ranges.index(r)
    assert all(0 <= w < warps for w in work)
    # The line counts a unit's keys / 32 rounded down, where its steps are rounded
    # up: a step more for each range at most. Where nothing is cut (units of at
    # most 8, as many as warps) a warp takes a unit; else a share, of 4 at least,
    # and a cut moves by a step and over a unit's fixed cost at each end.
    length = sum(max(w - 1, 0) + 2 for w in want.values())
    share = max(-(-(length + len(want)) // warps), 4, 8)
    for w, done in work.items():
        assert done <= share + sum(r["warp"] == w for r in ranges) + 2 * (1 + 2)


@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("h,h_kv,rows", [(4, 1, 8), (8, 8, 8), (16, 1, 16), (12, 4, 8), (5, 1, 16)])
@pytest.mark.parametrize("sq,sk", [
    ([1], [131072]), ([1], [1]), ([1], [0]), ([1, 1, 1], [1, 33, 4000]), ([4, 1, 2], [100, 2000, 1]),
    ([1] * 40, [1000] * 40), ([2, 0, 1], [50, 60, 0]), ([1, 9, 1], [300, 5000, 70]),
])
def test_plans(exattn_lib, sq, sk, h, h_kv, rows, causal):
    check(exattn_lib, sq, sk, h, h_kv, rows, causal, 2432 if rows == 8 else 1824)


def test_random_plans(exattn_lib):
    r = random.Random(7)
    for _ in range(150):
        b = r.choice([1, 2, 5, 33, 64, 100])
        most = r.choice([40, 900, 9000])
        sk = [r.randint(0, most) for _ in range(b)]
        sq = [r.choice([0, 1, 1, 1, 3]) for _ in range(b)]
        h_kv = r.choice([1, 2, 3, 8])
        check(exattn_lib, sq, sk, h_kv * r.choice([1, 2, 4, 7]), h_kv, r.choice([8, 16]), r.randrange(2),
              r.choice([7, 152, 1216, 2432]))


def test_refusals(exattn_lib):
    one = (ctypes.c_int * 1)(1)
    out = (ctypes.c_int * 90)()
    call = exattn_lib.attn_debug_few_plan
    assert call(None, one, 1, 4, 1, 8, 1, 9, 10, out) == -1
    assert call(one, one, 1, 4, 1, 9, 1, 9, 10, out) == -1
    assert call(one, one, 1, 16, 1, 8, 1, 9, 10, out) == -1
    assert call(one, one, 1, 5, 2, 8, 1, 9, 10, out) == -1
