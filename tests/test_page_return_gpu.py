"""A finished request's pages back on the free stack, on the device: its table's
entries behind the first free_count, the count raised by as many. The next step
takes them from the top, and results are those of a cache that never shared.
"""
import pytest
import torch

from packed_parity import check_forward, default_scale, fp32_slack, starts

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_pages_are_taken_again(gpu, oracle_mod):
    page, h, h_kv, d = 16, 4, 2, 64
    g = torch.Generator().manual_seed(3)
    pools = [torch.full((6, page, h_kv, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    table = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    free, count, lens = torch.arange(6, dtype=torch.int32, device="cuda"), ints([6]), ints([0, 0])

    def step(new):
        nonlocal lens, count
        rows = [torch.randn((sum(new), x, d), generator=g).bfloat16() for x in (h, h_kv, h_kv)]
        q, k, v = (x.cuda() for x in rows)
        cu, lens, slots, count = gpu.attn_paged_plan(lens, ints(new), table, free, count, page, max_tokens=sum(new))
        gpu.attn_paged_write(k, v, slots, *pools)
        o, lse = gpu.attn_chunk_paged(q, *pools, table, cu, lens, max_seqlen_q=max(new), causal=True)
        return rows, o, lse

    first, _, _ = step([40, 30])     # three pages and two: one is left
    assert count.item() == 1
    # request 0 is done: its three pages go back, without a look at the host
    at = torch.arange(4, device="cuda")
    used = at < (lens[0] + page - 1) // page
    spot = torch.where(used, count[0] + at, 5)
    free.scatter_(0, spot.long(), torch.where(used, table[0], free[5]))
    count = count + used.sum().to(torch.int32)
    lens = torch.where(torch.arange(2, device="cuda") == 0, 0, lens).to(torch.int32)
    assert count.item() == 4
    assert sorted(free[:4].tolist() + table[1, :2].tolist()) == list(range(6))
    rows, o, lse = step([50, 2])     # another request in its place: all four free pages, three of them old ones
    assert count.item() == 0 and lens.tolist() == [50, 32]
    q, new_k, new_v = rows
    keys, values = (torch.cat([x[:50], old[40:], x[50:]]) for x, old in ((new_k, first[1]), (new_v, first[2])))
    cq, ck, scale = starts([50, 2]), starts([50, 32]), default_scale(d)
    o_ref, l_ref = oracle_mod.packed_attention(q, keys, values, cq, ck, scale, True)
    a_ref, _ = oracle_mod.packed_attention(q, keys, values.abs(), cq, ck, scale, True)
    check_forward(o, lse, o_ref, l_ref, a_ref, torch.bfloat16, fp32_slack(q, keys, scale, d), 52)
    assert gpu.attn_get_device_status() == gpu.ATTN_OK
