"""How packed calls deal their work to CTAs, on the host (the kernels run the
same arithmetic): every unit's steps are covered exactly once, in order; the
CTAs that share a cut unit are neighbours and agree on who they are; no CTA
gets much more than its share.
"""
import ctypes
import random

import pytest

import exact_attention_65_gb300 as ea

FIELDS = ("cta", "seq", "head", "unit", "step0", "nstep", "slot", "first", "nparts")


def plan(lib, sq, sk, h, h_kv, one_tile, causal, by_key, ctas=152):
    b = len(sq)
    q = (ctypes.c_int * b)(*sq)
    k = (ctypes.c_int * b)(*sk)
    room = 1 << 18
    out = (ctypes.c_int * (9 * room))()
    n = lib.attn_debug_packed_plan(q, k, b, h, h_kv, one_tile, causal, by_key, ctas, room, out)
    assert 0 <= n < room
    return [dict(zip(FIELDS, out[9 * i:9 * i + 9])) for i in range(n)]


def steps_of(sq, sk, tokens, unit, one_tile, causal, by_key):
    """The steps a unit must visit, from the mask itself."""
    if not by_key:
        length = tokens * (1 if one_tile else 2)
        rows = range(unit * length, min((unit + 1) * length, sq))
        keys = max((min(sk, r + sk - sq + 1) if causal else sk) for r in rows)
        return 0, max(0, -(-keys // 128))
    keys = range(unit * 128, min((unit + 1) * 128, sk))
    every = -(-sq // tokens)
    first = max(0, keys[0] - (sk - sq)) // tokens if causal else 0
    first = min(first, every)
    return first, every - first


def check(lib, sq, sk, h, h_kv, one_tile, causal, by_key, ctas=152):
    tokens = 128 // (h // h_kv)
    ranges = plan(lib, sq, sk, h, h_kv, one_tile, causal, by_key, ctas)
    want = []
    for s, (n, m) in enumerate(zip(sq, sk)):
        length = 128 if by_key else tokens * (1 if one_tile else 2)
        for head in range(h_kv):
            for unit in range(-(-(m if by_key else n) // length)):
                want.append((s, head, unit))
    got, at = [], {}
    shares = {}
    for r in ranges:
        key = (r["seq"], r["head"], r["unit"])
        first, count = steps_of(sq[r["seq"]], sk[r["seq"]], tokens, r["unit"], one_tile, causal, by_key)
        if key not in at:
            got.append(key)
            at[key] = first
            assert r["step0"] == first
        assert r["step0"] == at[key], "a gap or an overlap"
        at[key] += r["nstep"]
        assert (r["slot"] == -1) == (r["nstep"] == count)
        if r["slot"] >= 0:
            assert r["nstep"] > 0
            assert r["slot"] == (1 if r["step0"] == first else 0)
            shares.setdefault(key, []).append(r)
        assert 0 <= r["cta"] < ctas
    assert got == want
    for key, end in at.items():
        first, count = steps_of(sq[key[0]], sk[key[0]], tokens, key[2], one_tile, causal, by_key)
        assert end == first + count
    used = set()
    for key, rs in shares.items():
        assert len(rs) == rs[0]["nparts"] >= 2
        for i, r in enumerate(rs):
            assert (r["first"], r["nparts"]) == (rs[0]["first"], len(rs))
            assert r["cta"] == r["first"] + i
            assert (r["slot"] == 1) == (i == 0)
            # a CTA's slots hold one range each
            assert (r["cta"], r["slot"]) not in used
            used.add((r["cta"], r["slot"]))
    return ranges


@pytest.mark.parametrize("by_key", [0, 1])
@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("h,h_kv", [(1, 1), (32, 8), (5, 1), (71, 1), (128, 1), (6, 2)])
def test_covers_every_step_once(exattn_lib, h, h_kv, causal, by_key):
    r = random.Random(h * 7 + causal + 2 * by_key)
    for trial in range(40):
        b = r.choice([1, 2, 3, 33, 70])
        top = r.choice([1, 5, 130, 700, 5000])
        sq = [r.choice([0, 1, r.randint(0, top)]) for _ in range(b)]
        kind = r.randrange(3)
        sk = [n if kind == 0 else (r.randint(0, top) if kind == 1 else n + r.randint(0, 3 * top)) for n in sq]
        check(exattn_lib, sq, sk, h, h_kv, r.randrange(2), causal, by_key, r.choice([1, 2, 7, 80, 152]))


def test_empty_batches_give_nothing(exattn_lib):
    assert plan(exattn_lib, [0, 0], [5, 0], 4, 2, 1, 1, 0) == []
    assert plan(exattn_lib, [3, 0], [0, 0], 4, 2, 1, 1, 1) == []


def test_one_long_cache_is_spread(exattn_lib):
    """One request, eight K/V heads: every CTA gets an equal share."""
    ranges = check(exattn_lib, [1], [32768], 32, 8, 1, 1, 0)
    load = {}
    for r in ranges:
        load[r["cta"]] = load.get(r["cta"], 0) + r["nstep"]
    assert len(load) == 152
    assert max(load.values()) <= -(-8 * 256 // 152) + 2


def test_long_prompts_are_balanced(exattn_lib):
    for by_key in (0, 1):
        ranges = check(exattn_lib, [8192, 7000], [8192, 7000], 32, 8, 0, 1, by_key)
        load = {}
        for r in ranges:
            load[r["cta"]] = load.get(r["cta"], 0) + r["nstep"]
        mean = sum(load.values()) / 152
        assert max(load.values()) <= 1.08 * mean


def test_small_units_are_not_cut(exattn_lib):
    """A unit for each CTA where they fit, whole."""
    ranges = check(exattn_lib, [150, 40, 90], [150, 40, 90], 16, 16, 0, 1, 0)
    assert all(r["slot"] == -1 for r in ranges)
    assert len({r["cta"] for r in ranges}) == len(ranges) == 48


def test_refuses_bad_arguments(exattn_lib):
    one = (ctypes.c_int * 1)(4)
    bad = (ctypes.c_int * 1)(-1)
    out = (ctypes.c_int * 9)()
    f = exattn_lib.attn_debug_packed_plan
    assert f(None, one, 1, 1, 1, 0, 0, 0, 152, 1, out) == -1
    assert f(one, bad, 1, 1, 1, 0, 0, 0, 152, 1, out) == -1
    assert f(one, one, 0, 1, 1, 0, 0, 0, 152, 1, out) == -1
    assert f(one, one, 1, 3, 2, 0, 0, 0, 152, 1, out) == -1
    assert f(one, one, 1, 129, 1, 0, 0, 0, 152, 1, out) == -1
    assert f(one, one, 1, 1, 1, 0, 0, 0, 0, 1, out) == -1
    assert ea.ATTN_OK == 0
