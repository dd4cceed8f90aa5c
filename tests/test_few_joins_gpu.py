"""Results of units that many warps share, joined in a CTA and in two levels
between CTAs. Calls with the same sizes and other queries come by turns: what a
join reads of an earlier call's partial results would be another call's.

(Read with plain loads instead of past L1, partial results of an earlier call came
out in 190 of 500 calls of the first shape and 250 to 300 of 400 of the third while
only a shuffle stood between the count of arrivals and the loads, in none with the
barrier.)
"""
import pytest
import torch

from packed_parity import starts
from test_chunk_q4_gpu import check, ints, make_cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("b,n,new,h,h_kv,d,page", [
    (3, 9000, 2, 8, 1, 32, 16),    # 16 rows, units over tens of CTAs
    (1, 30001, 1, 4, 1, 128, 16),  # 8 rows, one unit over all of them
    (8, 6000, 1, 16, 1, 128, 16),
    (2, 900, 1, 8, 2, 64, 48),     # units of a CTA or two
])
def test_calls_by_turns(gpu, oracle_mod, b, n, new, h, h_kv, d, page):
    lens = [n] * b
    kp, vp, table, k, v = make_cache(oracle_mod, lens, h_kv, d, page, 1.0, 1.0, n)
    g = torch.Generator().manual_seed(n + 1)
    queries = [torch.randn((b * new, h, d), generator=g).to(torch.bfloat16) for _ in range(4)]
    device = [q.cuda() for q in queries]
    args = (kp.cuda(), vp.cuda(), table.cuda(), ints(starts([new] * b)), ints(lens), new)
    want = [gpu.attn_chunk_paged_q4(q, *args, causal=True) for q in device]
    for q, (o, lse) in zip(queries[:2], want):
        check(o, lse, q, k, v, starts([new] * b), starts(lens), True, torch.bfloat16, oracle_mod)
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(300):
        o, lse = gpu.attn_chunk_paged_q4(device[i % 4], *args, causal=True)
        wrong += (o != want[i % 4][0]).any() | (lse != want[i % 4][1]).any()
    assert gpu.attn_get_device_status() == gpu.ATTN_OK
    assert wrong.item() == 0
