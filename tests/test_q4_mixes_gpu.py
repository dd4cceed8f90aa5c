"""Batches over a 4-bit cache that take both kernels, hints that are wrong or
missing, waits that run out, calls on the same workspace one behind the other,
and what a result's neighbours hold."""
import time

import numpy as np
import pytest
import torch

from packed_parity import starts
from test_chunk_q4_gpu import check, ints, make_cache, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("h,h_kv,d,dtype", [(8, 2, 128, torch.bfloat16), (4, 4, 64, torch.float16),
                                            (24, 2, 32, torch.bfloat16), (40, 2, 64, torch.float16),
                                            (9, 1, 128, torch.float16), (16, 1, 16, torch.bfloat16)])
def test_chunks_beside_few_rows(gpu, oracle_mod, h, h_kv, d, dtype, causal):
    new = [1, 70, 2, 0, 1, 300, 3, 9, 1, 17]
    lens = [900, 500, 1, 40, 0, 301, 2000, 9, 65, 100]
    run(gpu, oracle_mod, new, lens, h, h_kv, d, 16, dtype, causal)
    run(gpu, oracle_mod, new, lens, h, h_kv, d, 48, dtype, causal, hint=False, ks=0.3, vs=7.0)


def test_many_of_both(gpu, oracle_mod):
    r = np.random.default_rng(8)
    new = [int(x) for x in r.choice([0, 1, 1, 1, 2, 40], 90)]
    lens = [int(max(x, n)) for x, n in zip(r.integers(0, 700, 90), new)]
    run(gpu, oracle_mod, new, lens, 8, 2, 64, 16, torch.bfloat16)


@pytest.mark.parametrize("hint", [1, 2, 5, 16, 1 << 20, -3])
def test_hints_that_are_wrong(gpu, oracle_mod, hint):
    """max_seqlen_q picks a form; the results do not depend on it."""
    new, lens = [40, 1, 5, 130], [600, 333, 5, 130]
    for h, h_kv, d in ((8, 2, 128), (3, 3, 32), (16, 1, 64)):
        kp, vp, table, k, v = make_cache(oracle_mod, lens, h_kv, d, 16, 1.0, 1.0, 4)
        q = torch.randn((sum(new), h, d), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
        for causal in (True, False):
            o, lse = gpu.attn_chunk_paged_q4(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), ints(starts(new)),
                                             ints(lens), max_seqlen_q=hint, causal=causal)
            assert gpu.attn_get_device_status() == gpu.ATTN_OK
            check(o, lse, q, k, v, starts(new), starts(lens), causal, torch.bfloat16, oracle_mod)


@pytest.mark.parametrize("new", [[1, 1], [60, 1], [200]])
def test_skipped_loads_time_out_and_recover(gpu, oracle_mod, new):
    """Few rows, both kernels, the two-tile kernel: a status, not a hang, and the next call is right."""
    lens = [600, 500][:len(new)]
    kp, vp, table, k, v = make_cache(oracle_mod, lens, 2, 64, 16, 1.0, 1.0, 4)
    q = torch.randn((sum(new), 4, 64), generator=torch.Generator().manual_seed(3)).to(torch.float16)
    args = (q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), ints(starts(new)), ints(lens))
    assert gpu.attn_get_device_status() == gpu.ATTN_OK
    gpu.attn_debug_set_flags(gpu.ATTN_DEBUG_SKIP_LOADS)
    try:
        gpu.attn_chunk_paged_q4(*args, max_seqlen_q=max(new), causal=True)
    finally:
        gpu.attn_debug_set_flags(0)
    t0 = time.time()
    assert gpu.attn_get_device_status() == gpu.ATTN_ERR_DEVICE_TIMEOUT and time.time() - t0 < 60
    for _ in range(2):
        o, lse = gpu.attn_chunk_paged_q4(*args, max_seqlen_q=max(new), causal=True)
        assert gpu.attn_get_device_status() == gpu.ATTN_OK
        check(o, lse, q, k, v, starts(new), starts(lens), True, torch.float16, oracle_mod)


def test_calls_of_different_kinds_on_one_workspace(gpu, oracle_mod):
    """4-bit and 16-bit calls, few rows and chunks, by turns on one stream: each its own bits every time."""
    lens, news = [7000, 90, 2500], ([1, 1, 1], [1, 1, 300], [4, 4, 4], [100, 1, 7])
    kp, vp, table, k, v = make_cache(oracle_mod, lens, 2, 64, 16, 1.0, 1.0, 6)
    g = torch.Generator().manual_seed(1)
    pools = [torch.randn((kp.shape[0], 16, 2, 64), generator=g).to(torch.bfloat16).cuda() for _ in "kv"]
    calls = []
    for new in news:
        q = torch.randn((sum(new), 8, 64), generator=g).to(torch.bfloat16).cuda()
        rest = (table.cuda(), ints(starts(new)), ints(lens), max(new))
        calls.append(lambda q=q, rest=rest: gpu.attn_chunk_paged_q4(q, kp.cuda(), vp.cuda(), *rest, causal=True))
        calls.append(lambda q=q, rest=rest: gpu.attn_chunk_paged(q, *pools, *rest, causal=True))
    want = [call() for call in calls]
    for i in torch.randint(0, len(calls), (60,), generator=g).tolist():
        o, lse = calls[i]()
        assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])
    assert gpu.attn_get_device_status() == gpu.ATTN_OK


def test_results_read_right_behind_the_call(gpu, oracle_mod):
    """The kernels of a mixed batch overlap; what comes behind them in the stream sees both's results."""
    new, lens = [1] * 30 + [200, 64], [3000] * 32
    kp, vp, table, k, v = make_cache(oracle_mod, lens, 2, 64, 64, 1.0, 1.0, 2)
    q = torch.randn((sum(new), 8, 64), generator=torch.Generator().manual_seed(1)).to(torch.float16).cuda()
    out, lse = torch.empty_like(q), torch.empty((8, sum(new)), device="cuda")
    args = (q, kp.cuda(), vp.cuda(), table.cuda(), ints(starts(new)), ints(lens), 200)
    want = None
    for _ in range(50):
        out.fill_(7.0)
        lse.fill_(7.0)
        gpu.attn_chunk_paged_q4(*args, out=out, lse=lse, causal=True)
        got = out.clone(), lse.clone()
        if want is None:
            want = got
            check(*want, q.cpu(), k, v, starts(new), starts(lens), True, torch.float16, oracle_mod)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("page", [16, 64])
def test_values_of_nan_reach_their_own_rows_only(gpu, oracle_mod, page):
    """A scale of NaN in a request's own key turns the rows that see it to NaN, and no other."""
    lens, new = [300, 200, 80], [1, 3, 1]
    kp, vp, table, k, v = make_cache(oracle_mod, lens, 2, 64, page, 1.0, 1.0, 12)
    q = torch.randn((5, 4, 64), generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).cuda()
    args = (table.cuda(), ints(starts(new)), ints(lens))
    clean = gpu.attn_chunk_paged_q4(q, kp.cuda(), vp.cuda(), *args, 3, causal=True)
    # key 198 of request 1 (its last row but one sees it, the first does not), head 0
    slot = int(table[1, 198 // page]) * page + 198 % page
    for pool in (kp, vp):
        bad = pool.clone()
        bad[slot // page, 0, page * 32 + (slot % page) * 4] = 127
        o, lse = gpu.attn_chunk_paged_q4(q, *(bad.cuda() if x is pool else x.cuda() for x in (kp, vp)), *args, 3,
                                         causal=True)
        hit = torch.isnan(o.float()).any(-1)
        assert hit[[2, 3], :2].all() and not hit[[0, 1, 4]].any() and not hit[:, 2:].any()
        keep = ~hit
        assert torch.equal(o[keep], clean[0][keep])


@pytest.mark.parametrize("d,dtype", [(128, torch.bfloat16), (64, torch.float16), (16, torch.bfloat16)])
@pytest.mark.parametrize("key", [1, 255, 256, 399, 499])
def test_values_of_nan_in_a_chunk(gpu, oracle_mod, d, dtype, key):
    """The same of a chunk's rows, from the first that sees the key on, with a token of another request beside it."""
    lens, new, h, h_kv, page = [500, 90], [400, 1], 6, 2, 48
    kp, vp, table, k, v = make_cache(oracle_mod, lens, h_kv, d, page, 1.0, 1.0, 12)
    q = torch.randn((401, h, d), generator=torch.Generator().manual_seed(5)).to(dtype).cuda()
    args = (table.cuda(), ints(starts(new)), ints(lens))
    for hint in (400, 0):
        clean = gpu.attn_chunk_paged_q4(q, kp.cuda(), vp.cuda(), *args, hint, causal=True)
        slot = int(table[0, key // page]) * page + key % page
        for pool in (kp, vp):
            bad = pool.clone()
            bad[slot // page, 1, page * d // 2 + slot % page * (d // 16) + d // 16 - 1] = 127
            o, lse = gpu.attn_chunk_paged_q4(q, *(bad.cuda() if x is pool else x.cuda() for x in (kp, vp)), *args,
                                             hint, causal=True)
            assert gpu.attn_get_device_status() == gpu.ATTN_OK
            want = torch.zeros((401, h), dtype=torch.bool, device="cuda")
            want[max(key - 100, 0):400, 3:] = True  # row i of the chunk is token 100 + i
            assert torch.equal(torch.isnan(o.float()).any(-1), want)
            assert torch.equal(torch.isnan(lse).T, want)
            assert torch.equal(o[~want], clean[0][~want]) and torch.equal(lse.T[~want], clean[1].T[~want])


def test_another_device_index_and_wrong_shapes(gpu):
    """The binding's own refusals."""
    q = torch.zeros((2, 4, 64), dtype=torch.float16, device="cuda")
    pool = torch.zeros((3, 2, gpu.attn_q4_page_bytes(16, 64)), dtype=torch.uint8, device="cuda")
    cu, lens, table = ints([0, 1, 2]), ints([3, 3]), ints([[0], [1]])
    gpu.attn_chunk_paged_q4(q, pool, pool, table, cu, lens)
    for bad in (pool[:, :, :100].contiguous(), pool.to(torch.int8), pool[:, :1].contiguous().expand(3, 2, -1),
                pool.cpu(), pool[0]):
        with pytest.raises(ValueError):
            gpu.attn_chunk_paged_q4(q, bad, bad, table, cu, lens)
    with pytest.raises(ValueError):
        gpu.attn_chunk_paged_q4(q[:, :3].contiguous(), pool, pool, table, cu, lens)
    with pytest.raises(ValueError):
        gpu.attn_chunk_paged_q4(q, pool, pool, table.long(), cu, lens)
    with pytest.raises(gpu.AttnError):
        gpu.attn_chunk_paged_q4(q, pool, pool, table, cu, lens, k_scale=0.0)
    cs = torch.zeros((5, 64), device="cuda")
    n = ints([0, 1], torch.int64)
    k = q[:, :2].contiguous()
    gpu.attn_paged_append_q4(q, k, k, cs, n, n, pool, pool.clone())
    for kw in (dict(cos_sin=cs.double()), dict(positions=n.int()), dict(slot_map=n[:1]), dict(k=q), dict(k=k.float()),
               dict(k_pages=pool[:, :1].contiguous()), dict(q_out=q[:1])):
        args = dict(q=q, k=k, v=k, cos_sin=cs, positions=n, slot_map=n, k_pages=pool, v_pages=pool.clone())
        with pytest.raises((ValueError, TypeError)):
            gpu.attn_paged_append_q4(**{**args, **kw})
    with pytest.raises(gpu.AttnError):
        gpu.attn_paged_append_q4(q, k, k, cs[:, :24].contiguous(), n, n, pool, pool.clone())
    with pytest.raises(gpu.AttnError):  # (taken as pages of 8 rows)
        gpu.attn_paged_read_q4(pool, pool, n, 128)
    with pytest.raises(ValueError):
        gpu.attn_paged_read_q4(pool[:, :, :570].contiguous(), pool[:, :, :570].contiguous(), n, 64)
    with pytest.raises(ValueError):
        gpu.attn_paged_read_q4(pool, pool, n, 64, k=k[:1])
    with pytest.raises(TypeError):
        gpu.attn_paged_read_q4(pool, pool, n, 64, dtype=torch.float32)
