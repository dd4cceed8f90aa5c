"""Lengths, page numbers and starts over a 4-bit cache that lie outside what
the call's sizes say, on each of its kernels and on both at once: lengths and page
numbers are moved into their range, starts past the rows too, and starts out of
order leave the results as they were.
"""
import numpy as np
import pytest
import torch

from packed_parity import starts
from test_chunk_q4_gpu import check, ints

pytestmark = pytest.mark.gpu

H, H_KV, D = 8, 2, 64
FORMS = [  # new tokens, max_seqlen_q
    ([1, 1, 1], 1),      # 8 rows
    ([3, 1, 2], 3),      # 16 rows
    ([40, 70, 33], 70),  # two tiles
    ([1, 70, 2], 70),    # both kernels
    ([2, 40, 1], 0),
]


def whole_pool(oracle, pages, page, seed):
    """Pools in which every row is some token's: as bytes, and the values of all rows."""
    r = np.random.default_rng(seed)
    pools, values = [], []
    for _ in "kv":
        code, s = oracle.q4_quantise(r.standard_normal((pages * page, H_KV, D)), 1.0)
        pools.append(torch.from_numpy(oracle.q4_pool(code, s, pages, page)).cuda())
        values.append(oracle.q4_values(code, s, 1.0))
    return pools, values


def call(gpu, q, pools, table, cu, lens, hint, causal):
    """The call's results, with rows of sentinels behind them."""
    n = q.shape[0]
    out = torch.full((n + 3, H, D), 7.0, dtype=q.dtype, device="cuda")
    wide = torch.full((H + 2, n), 7.0, device="cuda")
    gpu.attn_chunk_paged_q4(q.cuda(), *pools, table, cu, lens, hint, out=out[:n], lse=wide[:H], causal=causal)
    assert gpu.attn_get_device_status() == gpu.ATTN_OK
    assert torch.all(out[n:] == 7) and torch.all(wide[H:] == 7)
    return out[:n], wide[:H]


def queries(n, seed=1):
    return torch.randn((n, H, D), generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


@pytest.mark.parametrize("new,hint", FORMS)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("page,width", [(16, 9), (48, 5)])
def test_lengths_and_pages(gpu, oracle_mod, new, hint, causal, page, width):
    pages = 7
    pools, (k, v) = whole_pool(oracle_mod, pages, page, 3)
    r = np.random.default_rng(9)
    table = r.integers(0, pages, (3, width))
    wild = [-1, pages, 10 ** 6, -2 ** 31, 2 ** 31 - 1]
    for i, x in enumerate(wild):
        table[i % 3, i] = x
    lens = [1 << 30, -5, width * page - 11]
    real = [width * page, 0, width * page - 11]
    q = queries(sum(new))
    o, lse = call(gpu, q, pools, ints(table), ints(starts(new)), ints(lens), hint, causal)
    at = np.concatenate([np.clip(table[i], 0, pages - 1)[np.arange(n) // page] * page + np.arange(n) % page
                         for i, n in enumerate(real)]).astype(int)
    check(o, lse, q, k[at], v[at], starts(new), starts(real), causal, torch.bfloat16, oracle_mod)


@pytest.mark.parametrize("new,hint", FORMS)
def test_starts_past_the_rows(gpu, oracle_mod, new, hint):
    """The last sequence has the rows that are there, and starts below 0 are 0."""
    pools, (k, v) = whole_pool(oracle_mod, 7, 16, 4)
    table, lens = np.arange(3)[:, None] * 2 + np.arange(2), [32, 20, 30]
    q = queries(sum(new))
    cu = starts(new)
    at = np.concatenate([table[i][np.arange(n) // 16] * 16 + np.arange(n) % 16 for i, n in enumerate(lens)])
    for bad in ([0, cu[1], cu[2], 10 ** 6], [-9, cu[1], cu[2], cu[3]], [-2 ** 31, cu[1], cu[2], 2 ** 31 - 1]):
        o, lse = call(gpu, q, pools, ints(table), ints(bad), ints(lens), hint, True)
        check(o, lse, q, k[at], v[at], cu, starts(lens), True, torch.bfloat16, oracle_mod)


@pytest.mark.parametrize("new,hint", FORMS)
def test_starts_out_of_order(gpu, oracle_mod, new, hint):
    """Nothing is dealt out, on either kernel, wherever the fault in the starts is."""
    pools, _ = whole_pool(oracle_mod, 7, 16, 5)
    table, lens = ints(np.arange(3)[:, None] * 2 + np.arange(2)), ints([32, 20, 30])
    n = sum(new)
    q = queries(n)
    cu = starts(new).tolist()
    for bad in ([0, 5 * n, cu[2], n], [0, cu[2], cu[1], n], [n, cu[1], cu[2], n], [0, cu[1], n, cu[2]],
                [0, cu[1], cu[2], -1]):
        o, lse = call(gpu, q, pools, table, ints(bad), lens, hint, True)
        assert torch.all(o == 7) and torch.all(lse == 7)


@pytest.mark.parametrize("new,hint", [([1] * 50, 1), ([1, 60] + [1] * 48, 60), ([40] * 50, 40)])
def test_starts_out_of_order_among_many(gpu, oracle_mod, new, hint):
    """More sequences than a warp has lanes: the line's sums tell."""
    pools, _ = whole_pool(oracle_mod, 7, 16, 6)
    table, lens = ints(np.arange(100).reshape(50, 2) % 7), ints([25] * 50)
    n = sum(new)
    for where in (1, 30, 33, 50):
        cu = starts(new)
        cu[where] = cu[where - 1] - 1
        o, lse = call(gpu, queries(n), pools, table, ints(cu), lens, hint, True)
        assert torch.all(o == 7) and torch.all(lse == 7)
