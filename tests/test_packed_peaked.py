"""Rows whose softmax sits on one key, in the packed backward: dS is near 0
there, and what rounding O puts into D = rowsum(dO O) would be most of it.

Rows that see few keys (at most 16) form D from P and dP in fp32. Their bound
leaves that rounding out. With u half a step of the type and s the largest sum
of |q k| scale over a row and a key, a score (d products) and the row's LSE (at
most 16 terms) are each off by at most f = (d + 16) 2^-23 (1 + s), which also
covers ex2 and lg2 (2^-22); dP is off by f |dO| |V|, P by 2 f P and D, a sum of
P dP, by 3 f sum_j P_j |dO| |V_j|:
    |ddS| <= (u + 3 f) |dS| + P (3 f sum_j P_j |dO| |V_j| + 2 f |dO| |V|^T),
and dQ, dK from it as there. The CPU tests show that D from the rounded O is
past this bound on the same inputs, so that it tells the two apart; longer
rows are held to packed_parity's bound, which allows for it.
"""
import numpy as np
import pytest
import torch

from packed_parity import check_backward, default_scale, fp32_slack, make, starts, unit_roundoff


def peaked(lens, d, seed, gap):
    """Inputs (h = h_kv = 2) in which each row of a sequence has one key whose
    score is `gap` above about 0."""
    q, k, v = make(lens, lens, 2, 2, d, torch.bfloat16, seed)
    cu = starts(lens)
    for a, z in zip(cu, cu[1:]):
        # keys of near-orthogonal directions; a row points along its own
        q[a:z] = (q[a:z].float() * 0.02).bfloat16()
        for i in range(a, z):
            x = k[a + (i * 7 + 3 - a) % (z - a)].float()
            q[i] = (q[i].float() + x * (gap / (x * x).sum(-1, keepdim=True) / default_scale(d))).bfloat16()
    dout = torch.randn(q.shape, generator=torch.Generator().manual_seed(seed + 9)).bfloat16()
    return q, k, v, dout, cu


def tight(q, k, v, dout, cu, causal):
    """Gradients in 64 bits, how far the kernel's may be, and what D from the
    rounded O makes of dQ and dK."""
    u, d, scale = unit_roundoff(torch.bfloat16), q.shape[2], default_scale(q.shape[2])
    Q, K, V, G = (x.double().numpy() for x in (q, k, v, dout))
    s = max(scale * (np.abs(Q[a:z, x]) @ np.abs(K[a:z, x]).T).max()
            for a, z in zip(cu, cu[1:]) for x in range(Q.shape[1]))
    f = (d + 16) * 2.0 ** -23 * (1 + s)
    grads, bounds, rough = ([np.zeros_like(Q) for _ in range(2)] for _ in range(3))
    for a, z in zip(cu, cu[1:]):
        for x in range(Q.shape[1]):
            qx, kx, vx, gx = Q[a:z, x], K[a:z, x], V[a:z, x], G[a:z, x]
            s = scale * (qx @ kx.T)
            if causal:
                s = np.where(np.tril(np.ones(s.shape, dtype=bool)), s, -np.inf)
            p = np.exp(s - s.max(axis=1, keepdims=True))
            p /= p.sum(axis=1, keepdims=True)
            dp, size = gx @ vx.T, np.abs(gx) @ np.abs(vx).T
            ds = p * (dp - (p * dp).sum(axis=1, keepdims=True))
            o = torch.tensor(p @ vx).bfloat16().double().numpy()
            ds_rough = p * (dp - (gx * o).sum(axis=1, keepdims=True))
            eds = (u + 3 * f) * np.abs(ds) + p * (3 * f * (p * size).sum(axis=1, keepdims=True) + 2 * f * size)
            for out, y in ((grads, ds), (rough, ds_rough)):
                out[0][a:z, x], out[1][a:z, x] = scale * (y @ kx), scale * (y.T @ qx)
            bounds[0][a:z, x], bounds[1][a:z, x] = scale * (eds @ np.abs(kx)), scale * (eds.T @ np.abs(qx))
    return grads, [b + u * np.abs(g) + 2.0 ** -24 for b, g in zip(bounds, grads)], rough


FEW = [([16] * 20, False), ([9, 16, 12, 2, 13, 1] * 4, False), ([16] * 20, True)]


@pytest.mark.parametrize("lens,causal", FEW)
def test_the_bound_tells_a_rounded_d_apart(lens, causal):
    q, k, v, dout, cu = peaked(lens, 16, 3, 9.0)
    grads, bounds, rough = tight(q, k, v, dout, cu, causal)
    for g, b, r in zip(grads, bounds, rough):
        assert (np.abs(r - g) > 3 * b).any()


@pytest.mark.gpu
@pytest.mark.parametrize("lens,causal", FEW)
def test_rows_of_few_keys(gpu, lens, causal):
    q, k, v, dout, cu = peaked(lens, 16, 3, 9.0)
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    dev = [x.cuda() for x in (q, k, v)]
    o, lse = gpu.attn_fwd_packed(*dev, c, c, causal=causal)
    got = gpu.attn_bwd_packed(*dev, o, lse, dout.cuda(), c, c, causal=causal)
    assert gpu.attn_get_device_status() == gpu.ATTN_OK
    grads, bounds, _ = tight(q, k, v, dout, cu, causal)
    for name, x, g, b in zip(("dq", "dk"), got, grads, bounds):
        err = np.abs(x.double().cpu().numpy() - g)
        assert (err <= b).all(), f"{name}: {(err / b).max():.2f} of its bound"


@pytest.mark.gpu
@pytest.mark.parametrize("d", [16, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_long_rows(gpu, oracle_mod, d, causal):
    q, k, v, dout, cu = peaked([400, 17, 130], d, 5, 9.0)
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    dev = [x.cuda() for x in (q, k, v)]
    o, lse = gpu.attn_fwd_packed(*dev, c, c, causal=causal)
    got = gpu.attn_bwd_packed(*dev, o, lse, dout.cuda(), c, c, causal=causal)
    assert gpu.attn_get_device_status() == gpu.ATTN_OK
    scale = default_scale(d)
    refs = oracle_mod.packed_attention_backward(q, k, v, dout, cu, cu, scale, causal)
    check_backward(got, q, k, v, o, dout, cu, cu, scale, causal, refs, torch.bfloat16, fp32_slack(q, k, scale, d))
