"""Results that a call makes itself lie in memory of the stream it runs on.
Memory that the current stream gave back may still be written there: here
every block that the results could take is, late, by work queued before.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def rows(*shape):
    return torch.randn(shape, device="cuda").bfloat16()


def cases(ea):
    q, k, v, g = (rows(2, 300, 4, 128) for _ in range(4))
    o, lse = ea.attn_fwd(q, k, v)
    yield "attn_fwd", lambda s: ea.attn_fwd(q, k, v, stream=s)
    yield "attn_bwd", lambda s: ea.attn_bwd(q, k, v, o, lse, g, stream=s)
    yield "attn_decode_splitkv", lambda s: ea.attn_decode_splitkv(q[:, :1].contiguous(), k, v, num_splits=2, stream=s)
    pools = [rows(40, 16, 4, 128) for _ in "kv"]
    table, lens = torch.arange(40, device="cuda", dtype=torch.int32).view(2, 20), ints([300, 77])
    one = q[:, :1].contiguous()
    yield "attn_decode_paged", lambda s: ea.attn_decode_paged(one, *pools, table, lens, stream=s)
    p = [x.flatten(0, 1) for x in (q, k, v, g)]
    cu = ints([0, 250, 600])
    po, pl = ea.attn_fwd_packed(*p[:3], cu, cu)
    yield "attn_fwd_packed", lambda s: ea.attn_fwd_packed(*p[:3], cu, cu, stream=s)
    yield "attn_bwd_packed", lambda s: ea.attn_bwd_packed(*p[:3], po, pl, p[3], cu, cu, stream=s)
    cq = ints([0, 1, 8])
    yield "attn_chunk_paged", lambda s: ea.attn_chunk_paged(p[0][:8], *pools, table, cq, lens, causal=True, stream=s)
    free, count, new = torch.arange(50, device="cuda", dtype=torch.int32), ints([50]), ints([5, 40])
    wide = torch.zeros(2, 30, device="cuda", dtype=torch.int32)
    yield "attn_paged_plan", lambda s: ea.attn_paged_plan(lens, new, wide, free, count, 16, max_tokens=50, stream=s)


NAMES = ["attn_fwd", "attn_bwd", "attn_decode_splitkv", "attn_decode_paged", "attn_fwd_packed", "attn_bwd_packed",
         "attn_chunk_paged", "attn_paged_plan"]


@pytest.mark.parametrize("name", NAMES)
def test_results_do_not_share_memory_still_in_use(gpu, name):
    torch.manual_seed(5)
    call = dict(cases(gpu))[name]
    want = [x.clone() for x in call(None)]
    sizes = sorted({x.numel() * x.element_size() for x in want})
    side = torch.cuda.Stream()
    for _ in range(3):
        call(side)  # (what a first call sets up is done)
    torch.cuda.synchronize()
    junk = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(6)]
    torch.cuda._sleep(40_000_000)  # some 20 ms
    for x in junk:
        x.fill_(119)
    taken = {x.data_ptr() for x in junk}
    del x, junk
    got = call(side)
    assert not taken & {x.data_ptr() for x in got}
    side.synchronize()
    torch.cuda.synchronize()
    assert gpu.attn_get_device_status() == gpu.ATTN_OK
    for x, y in zip(got, want):
        assert torch.equal(x, y)
