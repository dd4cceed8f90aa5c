"""How the packed backward shares its CTAs out between key tiles and query
tiles, on the host, also where a call is so large that a line counts its costs
in more than one step at a time.
"""
import ctypes

import pytest

from test_packed_plan import check


def shares(lib, sq, sk, h, h_kv, causal, ctas=152):
    b = len(sq)
    q, k, out = (ctypes.c_int * b)(*sq), (ctypes.c_int * b)(*sk), (ctypes.c_int * 2)()
    n = lib.attn_debug_packed_shares(q, k, b, h, h_kv, causal, ctas, out)
    assert 1 <= n < ctas
    return n, out[0], out[1]


def steps(sq, sk, group, causal):
    """Work of both kinds for one K/V head, in steps, by the mask: each unit's
    own and the two that its set-up counts as."""
    tokens = 128 // group
    q = kv = 0.0
    for n, m in zip(sq, sk):
        for u in range(-(-n // tokens)):
            last = min((u + 1) * tokens, n) - 1
            q += 2 + max(0, min(m, last + m - n + 1) if causal else m) / 128
        for u in range(-(-m // 128)):
            kv += 2 + max(0, n - max(0, u * 128 - (m - n) if causal else 0)) * group / 128
    return q, kv


@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("h,h_kv,b,total", [
    (32, 8, 1000, 600_000),    # both lines count single steps
    (32, 8, 1000, 655_000),    # the key line counts two at a time, the query line one
    (32, 8, 1000, 690_000),
    (32, 8, 1000, 800_000),    # both two
    (32, 8, 1000, 960_000),    # four, and two
    (32, 8, 64, 1_010_000),
    (16, 16, 300, 900_000),
    (8, 1, 2000, 2_000_000),
    (32, 8, 6, 16_456),
])
def test_shares_follow_the_work(exattn_lib, h, h_kv, b, total, causal):
    lens = [total // b + (1 if i < total % b else 0) for i in range(b)]
    n, _, _ = shares(exattn_lib, lens, lens, h, h_kv, causal)
    q, kv = steps(lens, lens, h // h_kv, causal)
    want = 152 * 1.15 * kv / (q + 1.15 * kv)
    # (the causal query units are counted up to a unit long, and the share is
    # rounded: a few CTAs; with different units for the two lines it would be
    # 25 of 152)
    assert abs(n - want) <= 6


def test_the_two_lines_may_count_in_different_units(exattn_lib):
    seen = set()
    for total in range(600_000, 1_000_001, 5_000):
        n, q, kv = shares(exattn_lib, [total // 1000] * 1000, [total // 1000] * 1000, 32, 8, 1)
        seen.add(kv - q)
        wq, wkv = steps([total // 1000], [total // 1000], 4, 1)
        assert abs(n - 152 * 1.15 * wkv / (wq + 1.15 * wkv)) <= 6
    assert seen == {0, 1}


@pytest.mark.parametrize("by_key", [0, 1])
@pytest.mark.parametrize("b,length,h,h_kv", [(1000, 660, 32, 8), (1, 1 << 20, 4, 4), (3, 300_000, 2, 1)])
def test_plans_counted_in_several_steps_at_a_time(exattn_lib, b, length, h, h_kv, by_key):
    check(exattn_lib, [length] * b, [length] * b, h, h_kv, 1, 1, by_key)
    check(exattn_lib, [length] * b, [length + 5] * b, h, h_kv, 0, 0, by_key)
