"""Packed forward (attn_fwd_packed) against the fp64 oracle: grouped heads,
ragged lengths (empty ones too), keys and rows of different counts, slices of
wider rows, rows behind the last sequence, NaN in rows of no sequence and in
neighbouring sequences, units cut over several CTAs, streams and graphs.
"""
import numpy as np
import pytest
import torch

from packed_parity import check_forward, default_scale, fp32_slack, make, starts

pytestmark = pytest.mark.gpu


def cuda(x):
    """On the device with the same strides."""
    if x.is_contiguous():
        return x.cuda()
    wide = torch.empty(x.shape[0], x.stride(0), dtype=x.dtype, device="cuda")
    y = wide[:, 8:8 + x.shape[1] * x.shape[2]].unflatten(1, x.shape[1:])
    y.copy_(x)
    return y


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def run(ea, oracle, lens_q, lens_k, h, h_kv, d, dtype, causal, seed=3, scale=None, tail=0, fused=False,
        hint=True):
    q, k, v = make(lens_q, lens_k, h, h_kv, d, dtype, seed, tail, fused)
    cq, ck = starts(lens_q), starts(lens_k)
    scale = default_scale(d) if scale is None else scale
    out = torch.full((q.shape[0], h, d), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((h, q.shape[0]), 7.0, device="cuda")
    ea.attn_fwd_packed(cuda(q), cuda(k), cuda(v), ints(cq), ints(ck), max_seqlen_q=max(lens_q) if hint else 0,
                       scale=scale, out=out, lse=lse, causal=causal)
    assert ea.attn_get_device_status() == ea.ATTN_OK
    n = int(cq[-1])
    o_ref, lse_ref = oracle.packed_attention(q, k, v, cq, ck, scale, causal)
    a_ref, _ = oracle.packed_attention(q, k, v.abs(), cq, ck, scale, causal)
    check_forward(out, lse, o_ref, lse_ref, a_ref, dtype, fp32_slack(q, k, scale, d), n)
    assert torch.all(out[n:] == 7.0) and torch.all(lse[:, n:] == 7.0), "rows of no sequence were written"


@pytest.mark.parametrize("h,h_kv", [(1, 1), (2, 2), (4, 1), (6, 2), (5, 1), (16, 2), (71, 1), (128, 1)])
@pytest.mark.parametrize("causal", [False, True])
def test_heads(gpu, oracle_mod, h, h_kv, causal):
    run(gpu, oracle_mod, [37, 1, 130], [37, 1, 130], h, h_kv, 64, torch.bfloat16, causal)


@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("causal", [False, True])
def test_head_dims(gpu, oracle_mod, d, dtype, causal):
    run(gpu, oracle_mod, [150, 7, 300], [150, 7, 300], 6, 2, d, dtype, causal)
    run(gpu, oracle_mod, [5, 1, 9], [500, 1, 77], 6, 2, d, dtype, causal)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens_q,lens_k", [
    ([0, 5, 0], [3, 5, 0]),           # empty sequences, keys nobody asks for
    ([4, 3], [0, 6]),                 # a sequence without keys
    ([1], [1]),
    ([200, 100], [50, 300]),          # more rows than keys (causal: rows that see none), and fewer
    ([128, 129, 127], [256, 257, 255]),
    ([1] * 40, list(range(1, 41))),
])
def test_lengths(gpu, oracle_mod, lens_q, lens_k, causal):
    run(gpu, oracle_mod, lens_q, lens_k, 8, 2, 128, torch.bfloat16, causal)


@pytest.mark.parametrize("hint", [False, True])
def test_many_short_sequences(gpu, oracle_mod, hint):
    r = np.random.default_rng(5)
    lens = [int(x) for x in r.integers(0, 90, 700)]
    run(gpu, oracle_mod, lens, lens, 4, 2, 32, torch.float16, True, hint=hint)


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("causal", [False, True])
def test_rows_of_no_sequence(gpu, oracle_mod, fused, causal):
    """NaN behind the last sequence, inside the last key tile."""
    run(gpu, oracle_mod, [70, 61], [70, 61], 4, 2, 128, torch.bfloat16, causal, tail=9, fused=fused)
    run(gpu, oracle_mod, [3, 2], [300, 130], 4, 2, 64, torch.float16, causal, tail=130, fused=fused)


@pytest.mark.parametrize("causal", [False, True])
def test_neighbours_do_not_leak(gpu, causal):
    """NaN and infinities in one sequence leave the others' bits alone."""
    lens = [100, 60, 90]
    q, k, v = (cuda(x) for x in make(lens, lens, 4, 2, 64, torch.bfloat16, 11))
    cu = ints(starts(lens))
    o, lse = gpu.attn_fwd_packed(q, k, v, cu, cu, causal=causal)
    for x, bad in ((q, float("nan")), (k, float("inf")), (v, float("nan"))):
        x[100:160] = bad
    o2, lse2 = gpu.attn_fwd_packed(q, k, v, cu, cu, causal=causal)
    assert gpu.attn_get_device_status() == gpu.ATTN_OK
    keep = torch.ones(250, dtype=torch.bool, device="cuda")
    keep[100:160] = False
    assert torch.equal(o[keep], o2[keep]) and torch.equal(lse[:, keep], lse2[:, keep])
    assert torch.isnan(o2[100:160]).all() and torch.isnan(lse2[:, 100:160]).all()


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("rows", [1, 3, 40, 700])
def test_cut_units(gpu, oracle_mod, rows, causal):
    """A long sequence beside short ones: its units are cut over many CTAs."""
    run(gpu, oracle_mod, [rows, 5, 1], [9000, 5, 700], 4, 1, 128, torch.bfloat16, causal)
    run(gpu, oracle_mod, [rows, 2], [5001, 300], 3, 3, 16, torch.float16, causal)


def test_same_bits_every_time(gpu):
    lens_q, lens_k = [600, 3], [9000, 4000]
    q, k, v = (cuda(x) for x in make(lens_q, lens_k, 8, 2, 128, torch.bfloat16, 13))
    cq, ck = ints(starts(lens_q)), ints(starts(lens_k))
    first = gpu.attn_fwd_packed(q, k, v, cq, ck, causal=True)
    for _ in range(20):
        again = gpu.attn_fwd_packed(q, k, v, cq, ck, causal=True)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("scale", [-0.3, 0.0, 2.0])
def test_scales(gpu, oracle_mod, scale):
    run(gpu, oracle_mod, [90, 33], [90, 133], 4, 2, 64, torch.bfloat16, True, scale=scale)


def test_wide_scores(gpu, oracle_mod):
    """Scores far apart: the running max moves late and the row sum spans many powers of two."""
    lens = [300]
    q, k, v = make(lens, lens, 2, 1, 64, torch.bfloat16, 17)
    k[200:] *= 12
    k[:100] *= -6
    cu = starts(lens)
    o, lse = gpu.attn_fwd_packed(cuda(q), cuda(k), cuda(v), ints(cu), ints(cu))
    o_ref, l_ref = oracle_mod.packed_attention(q, k, v, cu, cu, 0.125)
    a_ref, _ = oracle_mod.packed_attention(q, k, v.abs(), cu, cu, 0.125)
    check_forward(o, lse, o_ref, l_ref, a_ref, torch.bfloat16, fp32_slack(q, k, 0.125, 64), 300)


@pytest.mark.parametrize("causal", [False, True])
def test_matches_the_dense_forward(gpu, causal):
    """Equal lengths and a K/V head for each head: as attn_fwd, within two roundings."""
    b, s, h, d = 3, 260, 4, 128
    q, k, v = (torch.randn(b, s, h, d, device="cuda", dtype=torch.bfloat16) for _ in range(3))
    o, lse = gpu.attn_fwd(q, k, v, causal=causal)
    cu = ints([0, s, 2 * s, 3 * s])
    o2, lse2 = gpu.attn_fwd_packed(*(x.flatten(0, 1) for x in (q, k, v)), cu, cu, causal=causal)
    assert torch.allclose(lse.permute(1, 0, 2).reshape(h, -1), lse2, atol=2e-6, rtol=0)
    assert (o.flatten(0, 1).float() - o2.float()).abs().max() <= 2 ** -7 * v.float().abs().max()


def test_clamps_starts_that_are_out_of_range(gpu):
    """Rows outside the tensors are never touched, whatever the starts say."""
    q, k, v = (torch.randn(64, 2, 64, device="cuda", dtype=torch.float16) for _ in range(3))
    for cu in ([0, 100, 64], [-5, 30, 10 ** 9], [64, 10, 64], [0, 2 ** 31 - 1, 0]):
        out = torch.full((66, 2, 64), 7.0, device="cuda", dtype=torch.float16)
        gpu.attn_fwd_packed(q, k, v, ints(cu), ints(cu), out=out[1:65], causal=True)
        assert gpu.attn_get_device_status() == gpu.ATTN_OK
        assert torch.all(out[0] == 7.0) and torch.all(out[65] == 7.0)


def test_other_stream_and_graphs(gpu, oracle_mod):
    """Another stream; a graph replayed with new inputs and lengths; two graphs
    with cut units at work at the same time."""
    lens = [2, 1]
    keys = [9000, 300]
    sets = []
    for seed in (1, 2):
        q, k, v = make(lens, keys, 8, 2, 64, torch.bfloat16, seed)
        want, _ = oracle_mod.packed_attention(q, k, v, starts(lens), starts(keys), 0.125, True)
        sets.append(([cuda(x) for x in (q, k, v)], want))
    cq, ck = ints(starts(lens)), ints(starts(keys))
    side = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs, graphs = [], []
    for (qkv, _), s in zip(sets, side):
        o, lse = gpu.attn_fwd_packed(*qkv, cq, ck, stream=s, causal=True)
        s.synchronize()
        out, l2 = torch.empty_like(o), torch.empty_like(lse)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            gpu.attn_fwd_packed(*qkv, cq, ck, max_seqlen_q=2, out=out, lse=l2, causal=True)
        outs.append((o, lse, out, l2))
        graphs.append(graph)
    for _ in range(20):
        for graph, s in zip(graphs, side):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    assert gpu.attn_get_device_status() == gpu.ATTN_OK
    for (o, lse, out, l2), (_, want) in zip(outs, sets):
        assert torch.allclose(lse, l2, atol=1e-5, rtol=0)
        assert (out.double().cpu().numpy() - want).__abs__().max() < 2 ** -7 * 5
        assert (out.float() - o.float()).abs().max() < 2 ** -7 * 5
    # the same graph with other keys in the same place
    sets[0][0][1].copy_(sets[1][0][1])
    sets[0][0][2].copy_(sets[1][0][2])
    graphs[0].replay()
    eager, _ = gpu.attn_fwd_packed(*sets[0][0], cq, ck, max_seqlen_q=2, causal=True)
    assert torch.equal(outs[0][2], eager)


def test_a_call_that_gave_up_leaves_nothing_behind(gpu, oracle_mod):
    """A timeout between two calls with cut units: the next result is right."""
    lens, keys = [1], [9000]
    q, k, v = make(lens, keys, 4, 1, 128, torch.bfloat16, 23)
    args = [cuda(x) for x in (q, k, v)] + [ints(starts(lens)), ints(starts(keys))]
    first, _ = gpu.attn_fwd_packed(*args)
    gpu.attn_debug_set_flags(gpu.ATTN_DEBUG_SKIP_LOADS)
    try:
        gpu.attn_fwd_packed(*args)
    finally:
        gpu.attn_debug_set_flags(0)
    assert gpu.attn_get_device_status() == gpu.ATTN_ERR_DEVICE_TIMEOUT
    assert gpu.attn_last_timeout_site() >> 8 == 1
    again, _ = gpu.attn_fwd_packed(*args)
    assert gpu.attn_get_device_status() == gpu.ATTN_OK
    assert torch.equal(first, again)
