"""Shared by the packed and paged tests: inputs, and how far results may be
from the fp64 oracle.

Bounds, with u = eps / 2 of the 16-bit type (half a step, relative):
  O    is a sum of p_j v_j whose weights were rounded once (each off by at
       most u p_j) and is rounded once itself:  |dO| <= u (A + |O|), A = sum_j
       p_j |v_j|; the fp32 steps (products of d terms, ex2, sums) are below
       f (A + |O|), f = (d + 64) 2^-23 (1 + s), s the largest sum of |q k| scale.
  LSE  only has fp32 steps: |dLSE| <= f.
"""
import math

import numpy as np
import torch


def starts(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)


def make(lens_q, lens_k, h, h_kv, d, dtype, seed, tail=0, fused=False):
    """Host tensors q [tq + tail, h, d], k, v [tk + tail, h_kv, d]; fused: slices
    of wider rows. Rows behind the last sequence hold NaN."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for total, heads in ((sum(lens_q), h), (sum(lens_k), h_kv), (sum(lens_k), h_kv)):
        wide = torch.full((total + tail, heads * d + (24 if fused else 0)), float("nan"), dtype=dtype)
        wide[:total] = torch.randn((total, wide.shape[1]), generator=g).to(dtype)
        x = wide[:, 8:8 + heads * d] if fused else wide
        out.append(x.unflatten(1, (heads, d)))
    return out


def unit_roundoff(dtype):
    return torch.finfo(dtype).eps / 2


def fp32_slack(q, k, scale, d):
    """f of the module's text."""
    qa = np.nan_to_num(np.abs(q.double().numpy())).max(axis=(0, 1), initial=0.0)
    ka = np.nan_to_num(np.abs(k.double().numpy())).max(axis=(0, 1), initial=0.0)
    return (d + 64) * 2.0 ** -23 * (1.0 + abs(scale) * float(qa @ ka))


def check_forward(o, lse, o_ref, lse_ref, a_ref, dtype, slack, rows):
    """o [t, h, d], lse [h, t] (device) against the oracle over the first
    ``rows`` rows; a_ref is the oracle's output for |v|."""
    o64, l64 = o.double().cpu().numpy()[:rows], lse.double().cpu().numpy()[:, :rows]
    o_ref, lse_ref, a_ref = o_ref[:rows], lse_ref[:, :rows], a_ref[:rows]
    seen = np.isfinite(lse_ref)
    assert np.all(np.isneginf(l64[~seen])), "a row without a key: LSE = -inf"
    assert np.all(o64.transpose(1, 0, 2)[~seen] == 0.0), "a row without a key: O = 0"
    assert np.all(np.isfinite(o64)) and np.all(np.isfinite(l64[seen]))
    bound = (unit_roundoff(dtype) + slack) * (a_ref + np.abs(o_ref)) + 2.0 ** -24
    bad = np.abs(o64 - o_ref) - bound
    assert bad.max(initial=-1.0) <= 0, f"O off by {np.abs(o64 - o_ref).max():.3e}, {bad.max():.3e} over its bound"
    err = np.abs(l64[seen] - lse_ref[seen]).max(initial=0.0)
    assert err <= slack, f"LSE off by {err:.3e} > {slack:.3e}"


def default_scale(d):
    return 1.0 / math.sqrt(d)


def check_backward(grads, q, k, v, o, dout, cq, ck, scale, causal, refs, dtype, slack):
    """(dq, dk, dv) (device) against the oracle's. Per sequence and head, with P
    the weights and u, f as above:
      P and dS are rounded once before the products that add them up, D is
      the row sum of dO times the rounded O, and each result is rounded:
        |ddV| <= (u + f) P^T |dO| + u |dV|
        |ddS| <= (u + f) |dS| + P (e + 2 f |dO| |V|^T),  e = (u + f) rowsum(|dO| (A + |O|))
        |ddQ| <= scale |ddS| |K| + u |dQ|,  |ddK| <= scale |ddS|^T |Q| + u |dK|."""
    u, f = unit_roundoff(dtype), slack
    got = [x.double().cpu().numpy() for x in grads]
    Q, K, V, O, G = (x.double().cpu().numpy() for x in (q, k, v, o, dout))
    h, group = Q.shape[1], Q.shape[1] // K.shape[1]
    bounds = [u * np.abs(r) + 2.0 ** -24 for r in refs]
    for i in range(len(cq) - 1):
        a, z, ka, kz = (int(x) for x in (cq[i], cq[i + 1], ck[i], ck[i + 1]))
        if z == a or kz == ka:
            continue
        hidden = np.arange(kz - ka)[None] > np.arange(z - a)[:, None] + (kz - ka) - (z - a)
        for x in range(h):
            y = x // group
            qx, gx, kx, vx = Q[a:z, x], G[a:z, x], K[ka:kz, y], V[ka:kz, y]
            s = scale * (qx @ kx.T)
            if causal:
                s = np.where(hidden, -np.inf, s)
            m = s.max(axis=1, keepdims=True)
            p = np.exp(s - np.where(np.isfinite(m), m, 0.0))
            total = p.sum(axis=1, keepdims=True)
            p = p / np.where(total > 0, total, 1.0)
            dp = gx @ vx.T
            ds = np.abs(p * (dp - (p * dp).sum(axis=1, keepdims=True)))
            e = (u + f) * (np.abs(gx) * (p @ np.abs(vx) + np.abs(O[a:z, x]))).sum(axis=1, keepdims=True)
            eds = (u + f) * ds + p * (e + 2 * f * (np.abs(gx) @ np.abs(vx).T))
            bounds[0][a:z, x] += abs(scale) * (eds @ np.abs(kx))
            bounds[1][ka:kz, y] += abs(scale) * (eds.T @ np.abs(qx))
            bounds[2][ka:kz, y] += (u + f) * (p.T @ np.abs(gx))
    for name, x, ref, bound in zip(("dq", "dk", "dv"), got, refs, bounds):
        rows = int(cq[-1] if name == "dq" else ck[-1])
        x, ref, bound = x[:rows], ref[:rows], bound[:rows]
        assert np.all(np.isfinite(x)), f"{name} is not finite"
        over = (np.abs(x - ref) - bound).max(initial=-1.0)
        assert over <= 0, f"{name} off by {np.abs(x - ref).max():.3e}, {over:.3e} over its bound"
