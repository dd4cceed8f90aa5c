"""Packed backward (attn_bwd_packed) against the fp64 oracle's chain rule:
grouped heads (gradients of a shared K/V head are sums), ragged lengths, slices
of wider rows for inputs and gradients, NaN in rows of no sequence, cut units,
streams and graphs; and a training step with the forward.
"""
import numpy as np
import pytest
import torch

from packed_parity import check_backward, default_scale, fp32_slack, make, starts
from test_packed_gpu import cuda, ints

pytestmark = pytest.mark.gpu


def wide_like(x, fill):
    """A slice of wider rows with x's shape, everything filled."""
    rows = torch.full((x.shape[0], x.shape[1] * x.shape[2] + 24), fill, dtype=x.dtype, device="cuda")
    return rows, rows[:, 16:16 + x.shape[1] * x.shape[2]].unflatten(1, x.shape[1:])


def run(ea, oracle, lens_q, lens_k, h, h_kv, d, dtype, causal, seed=3, scale=None, tail=0, fused=False):
    q, k, v = make(lens_q, lens_k, h, h_kv, d, dtype, seed, tail, fused)
    cq, ck = starts(lens_q), starts(lens_k)
    scale = default_scale(d) if scale is None else scale
    g = torch.Generator().manual_seed(seed + 50)
    n, m = int(cq[-1]), int(ck[-1])
    dout = torch.full((n + tail, h, d), float("nan"), dtype=dtype)
    dout[:n] = torch.randn((n, h, d), generator=g).to(dtype)
    dev = [cuda(x) for x in (q, k, v)]
    # rows of no sequence of o and lse are whatever their buffers held
    o = torch.full((n + tail, h, d), float("nan"), dtype=dtype, device="cuda")
    lse = torch.full((h, n + tail), float("nan"), device="cuda")
    ea.attn_fwd_packed(*dev, ints(cq), ints(ck), scale=scale, out=o, lse=lse, causal=causal)
    if fused:
        wide = [wide_like(x, 7.0) for x in (q, k, v)]
        outs = [x[1] for x in wide]
    else:
        outs = [torch.full(x.shape, 7.0, dtype=dtype, device="cuda") for x in (q, k, v)]
    ea.attn_bwd_packed(*dev, o, lse, dout.cuda(), ints(cq), ints(ck), scale=scale, dq=outs[0], dk=outs[1],
                       dv=outs[2], causal=causal)
    assert ea.attn_get_device_status() == ea.ATTN_OK
    refs = oracle.packed_attention_backward(q[:n], k[:m], v[:m], dout[:n], cq, ck, scale, causal)
    check_backward([x[:r] for x, r in zip(outs, (n, m, m))], q[:n], k[:m], v[:m], o[:n], dout[:n], cq, ck, scale,
                   causal, refs, dtype, fp32_slack(q, k, scale, d))
    for x, r in zip(outs, (n, m, m)):
        assert torch.all(x[r:] == 7.0), "rows of no sequence were written"
    if fused:
        for (rows, _), x in zip(wide, (q, k, v)):
            width = x.shape[1] * x.shape[2]
            assert torch.all(rows[:, :16] == 7.0) and torch.all(rows[:, 16 + width:] == 7.0)


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
    ([0, 5, 0], [3, 5, 0]),           # keys nobody asks for: their gradients are 0
    ([4, 3], [0, 6]),                 # rows without keys
    ([1], [1]),
    ([200, 100], [50, 300]),
    ([128, 129, 127], [256, 257, 255]),
    ([1] * 40, list(range(1, 41))),
    ([0, 0, 0, 9], [200, 1, 300, 9]),
])
def test_lengths(gpu, oracle_mod, lens_q, lens_k, causal):
    run(gpu, oracle_mod, lens_q, lens_k, 8, 2, 128, torch.bfloat16, causal)


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("causal", [False, True])
def test_rows_of_no_sequence(gpu, oracle_mod, fused, causal):
    run(gpu, oracle_mod, [70, 61], [70, 61], 4, 2, 128, torch.bfloat16, causal, tail=9, fused=fused)
    run(gpu, oracle_mod, [3, 2], [300, 130], 4, 2, 64, torch.float16, causal, tail=130, fused=fused)


@pytest.mark.parametrize("causal", [False, True])
def test_neighbours_do_not_leak(gpu, causal):
    """NaN and infinities in one sequence leave the others' gradients alone."""
    lens = [100, 60, 90]
    q, k, v = (cuda(x) for x in make(lens, lens, 5, 1, 64, torch.bfloat16, 11))
    dout = torch.randn_like(q)
    cu = ints(starts(lens))
    o, lse = gpu.attn_fwd_packed(q, k, v, cu, cu, causal=causal)
    first = gpu.attn_bwd_packed(q, k, v, o, lse, dout, cu, cu, causal=causal)
    for x, bad in ((q, float("nan")), (k, float("inf")), (v, float("nan")), (dout, float("inf"))):
        x[100:160] = bad
    o, lse = gpu.attn_fwd_packed(q, k, v, cu, cu, causal=causal)
    second = gpu.attn_bwd_packed(q, k, v, o, lse, dout, cu, cu, causal=causal)
    assert gpu.attn_get_device_status() == gpu.ATTN_OK
    keep = torch.ones(250, dtype=torch.bool, device="cuda")
    keep[100:160] = False
    for x, y in zip(first, second):
        assert torch.equal(x[keep], y[keep])
        assert torch.isnan(y[100:160]).any()


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("h,h_kv,rows,keys", [(4, 1, 1500, 1500), (1, 1, 40, 6000), (2, 2, 3000, 100)])
def test_cut_units(gpu, oracle_mod, h, h_kv, rows, keys, causal):
    run(gpu, oracle_mod, [rows, 5], [keys, 5], h, h_kv, 64, torch.bfloat16, causal)
    run(gpu, oracle_mod, [rows, 5], [keys, 5], h, h_kv, 16, torch.float16, causal)


@pytest.mark.parametrize("scale", [-0.3, 0.0])
def test_scales(gpu, oracle_mod, scale):
    run(gpu, oracle_mod, [90, 33], [90, 133], 4, 2, 64, torch.bfloat16, True, scale=scale)


def test_many_short_sequences(gpu, oracle_mod):
    r = np.random.default_rng(5)
    lens = [int(x) for x in r.integers(0, 90, 400)]
    run(gpu, oracle_mod, lens, lens, 4, 2, 32, torch.float16, True)


def test_same_bits_every_time_and_graph(gpu):
    lens = [700, 3, 1200]
    q, k, v = (cuda(x) for x in make(lens, lens, 8, 2, 128, torch.bfloat16, 13))
    dout = torch.randn_like(q)
    cu = ints(starts(lens))

    def step(out=None):
        o, lse = gpu.attn_fwd_packed(q, k, v, cu, cu, causal=True)
        grads = out or [torch.empty_like(x) for x in (q, k, v)]
        gpu.attn_bwd_packed(q, k, v, o, lse, dout, cu, cu, dq=grads[0], dk=grads[1], dv=grads[2], causal=True)
        return grads

    first = step()
    for _ in range(10):
        assert all(torch.equal(x, y) for x, y in zip(first, step()))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        assert all(torch.equal(x, y) for x, y in zip(first, step()))
    s.synchronize()
    outs = [torch.empty_like(x) for x in (q, k, v)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(outs)
    for _ in range(3):
        for x in outs:
            x.fill_(7.0)
        graph.replay()
        assert all(torch.equal(x, y) for x, y in zip(first, outs))
    assert gpu.attn_get_device_status() == gpu.ATTN_OK


def test_skipped_loads_time_out_and_recover(gpu):
    lens = [900, 900]
    q, k, v = (cuda(x) for x in make(lens, lens, 4, 1, 128, torch.bfloat16, 13))
    cu = ints(starts(lens))
    o, lse = gpu.attn_fwd_packed(q, k, v, cu, cu, causal=True)
    args = (q, k, v, o, lse, torch.randn_like(q), cu, cu)
    first = gpu.attn_bwd_packed(*args, causal=True)
    gpu.attn_debug_set_flags(gpu.ATTN_DEBUG_SKIP_LOADS)
    try:
        gpu.attn_bwd_packed(*args, causal=True)
    finally:
        gpu.attn_debug_set_flags(0)
    assert gpu.attn_get_device_status() == gpu.ATTN_ERR_DEVICE_TIMEOUT
    assert gpu.attn_last_timeout_site() >> 8 == 3
    again = gpu.attn_bwd_packed(*args, causal=True)
    assert gpu.attn_get_device_status() == gpu.ATTN_OK
    assert all(torch.equal(x, y) for x, y in zip(first, again))


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens", [[1] * 60, [1] * 60 + [2], [2, 3, 9, 17]])
def test_rows_of_few_keys(gpu, oracle_mod, lens, causal):
    """A row with one key has dS = 0: rounding O must not leave noise in dQ and dK."""
    q, k, v = make(lens, lens, 4, 2, 64, torch.bfloat16, 41)
    cu = starts(lens)
    n = int(cu[-1])
    dout = torch.randn((n, 4, 64), generator=torch.Generator().manual_seed(5)).bfloat16()
    dev = [x.cuda() for x in (q, k, v)]
    o, lse = gpu.attn_fwd_packed(*dev, ints(cu), ints(cu), causal=causal)
    grads = gpu.attn_bwd_packed(*dev, o, lse, dout.cuda(), ints(cu), ints(cu), causal=causal)
    assert gpu.attn_get_device_status() == gpu.ATTN_OK
    refs = oracle_mod.packed_attention_backward(q, k, v, dout, cu, cu, 0.125, causal)
    # one key: P = 1, dP = D; P is off by f (the LSE's bound) and D by f |dO| |V|
    f = fp32_slack(q, k, 0.125, 64)
    one = np.repeat([m == 1 for m in lens], lens)
    size = (dout.abs().double().numpy() * np.repeat(v.abs().double().numpy(), 2, axis=1)).sum(-1).max()
    for x, like in zip(grads[:2], (k, q)):
        noise = np.abs(x.double().cpu().numpy()[one]).max(initial=0.0)
        assert noise <= 2 * 0.125 * 3 * f * size * float(like.abs().max())
    for x, r in zip(grads, refs):
        r = r[~one]
        if r.size and np.linalg.norm(r) > 0:
            got = x.double().cpu().numpy()[~one]
            assert np.linalg.norm(got - r) <= 3 * 2.0 ** -8 * np.linalg.norm(r)


def test_binding_refuses(gpu):
    q = torch.zeros(8, 4, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(8, 2, 64, dtype=torch.bfloat16, device="cuda")
    cu = ints([0, 8])
    o, lse = gpu.attn_fwd_packed(q, k, k, cu, cu)
    bad = [
        dict(k=k.half()), dict(k=k[:, :, :32]), dict(v=k[:4]), dict(cu_seqlens_q=cu.long()),
        dict(cu_seqlens_k=ints([0, 4, 8])), dict(q=q.transpose(0, 1)), dict(q=q[0]), dict(k=k.expand(8, 2, 64)[:, :1]),
        dict(out=o[:4]), dict(lse=lse.half()), dict(out=torch.zeros(8, 4, 128, device="cuda").bfloat16()[:, :, ::2]),
    ]
    for kw in bad:
        args = dict(dict(q=q, k=k, v=k, cu_seqlens_q=cu, cu_seqlens_k=cu), **kw)
        if kw.keys() == {"k"} and args["k"].shape[1] == 1:
            args["v"] = k  # shapes differ
        with pytest.raises((ValueError, TypeError)):
            gpu.attn_fwd_packed(**args)
    for kw in (dict(dout=q[:4]), dict(dout=torch.zeros(8, 4, 128, device="cuda").bfloat16()[:, :, ::2]),
               dict(dq=k), dict(dk=k.half()), dict(o=None), dict(lse=None)):
        args = dict(dict(q=q, k=k, v=k, o=o, lse=lse, dout=q, cu_seqlens_q=cu, cu_seqlens_k=cu), **kw)
        with pytest.raises((ValueError, TypeError)):
            gpu.attn_bwd_packed(**args)
    # heads that do not divide, and too many for one K/V head
    with pytest.raises(ValueError):
        gpu.attn_fwd_packed(q[:, :3].contiguous(), k, k, cu, cu)
    many = torch.zeros(8, 129, 16, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(gpu.AttnError):
        gpu.attn_fwd_packed(many, many[:, :1].contiguous(), many[:, :1].contiguous(), cu, cu)
