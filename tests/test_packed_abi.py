"""Refusals of the packed and paged entry points, and pins of their oracle; no GPU.

The C ABI checks its arguments before any pointer is used, so invalid calls
are made here with addresses that are never dereferenced.
"""
import numpy as np
import pytest
import torch

import exact_attention_65_gb300 as ea

A = 0x10000  # 16-byte aligned, never dereferenced
INV, UNS = ea.ATTN_ERR_INVALID_ARG, ea.ATTN_ERR_UNSUPPORTED


def call(fn, order, **kw):
    return fn(*[kw[x] for x in order.split()])


FWD = "q k v cq ck o lse b tq tk mq h hk d qs ks vs scale causal dtype stream"
FWD_OK = dict(q=A, k=A, v=A, cq=A, ck=A, o=A, lse=A, b=2, tq=10, tk=10, mq=0, h=4, hk=2, d=64, qs=256, ks=128,
              vs=128, scale=0.1, causal=1, dtype=ea.ATTN_BF16, stream=None)


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), INV), (dict(cq=None), INV), (dict(ck=None), INV), (dict(lse=None), INV),
    (dict(k=A + 8), INV), (dict(o=A + 2), INV), (dict(lse=A + 2), INV), (dict(cq=A + 1), INV),
    (dict(b=0), INV), (dict(tq=0), INV), (dict(tk=0), INV), (dict(h=0), INV), (dict(hk=0), INV),
    (dict(h=5), INV), (dict(scale=float("nan")), INV), (dict(dtype=7), INV),
    (dict(qs=255), INV), (dict(qs=248), INV), (dict(ks=132), INV), (dict(vs=64), INV),
    (dict(d=48), UNS), (dict(d=256), UNS), (dict(b=70000), UNS), (dict(h=258, hk=2, qs=1 << 15), UNS),
    (dict(tq=0x7fffffff), UNS), (dict(tk=0x7fffffff), UNS), (dict(qs=1 << 40), UNS),
])
def test_fwd_packed_refuses(exattn_lib, kw, expect):
    assert call(exattn_lib.attn_fwd_packed, FWD, **{**FWD_OK, **kw}) == expect


BWD = "q k v o lse do cq ck dq dk dv b tq tk h hk d qs ks vs dqs dks dvs scale causal dtype stream"
BWD_OK = dict(FWD_OK, do=A, dq=A, dk=A, dv=A, dqs=256, dks=128, dvs=128)


@pytest.mark.parametrize("kw,expect", [
    (dict(do=None), INV), (dict(dq=None), INV), (dict(dv=A + 8), INV), (dict(lse=None), INV), (dict(ck=A + 2), INV),
    (dict(dqs=128), INV), (dict(dks=129), INV), (dict(dvs=0), INV), (dict(tk=0), INV), (dict(h=3), INV),
    (dict(d=8), UNS), (dict(h=258, hk=2, qs=1 << 15, dqs=1 << 15), UNS),
])
def test_bwd_packed_refuses(exattn_lib, kw, expect):
    assert call(exattn_lib.attn_bwd_packed, BWD, **{**BWD_OK, **kw}) == expect


CHUNK = "q kp vp table cq lens o lse b tq mq h hk d pages page width qs scale causal dtype stream"
CHUNK_OK = dict(FWD_OK, kp=A, vp=A, table=A, lens=A, pages=9, page=16, width=4)


@pytest.mark.parametrize("kw,expect", [
    (dict(kp=None), INV), (dict(table=None), INV), (dict(lens=None), INV), (dict(vp=A + 8), INV),
    (dict(table=A + 2), INV), (dict(pages=0), INV), (dict(page=0), INV), (dict(width=0), INV), (dict(h=6, hk=4), INV),
    (dict(qs=64), INV), (dict(page=24), UNS), (dict(page=8), UNS), (dict(d=96), UNS),
    (dict(page=1 << 20, width=1 << 12), UNS),
])
def test_chunk_paged_refuses(exattn_lib, kw, expect):
    assert call(exattn_lib.attn_chunk_paged, CHUNK, **{**CHUNK_OK, **kw}) == expect


PLAN = "lens new table free count cq out slots left b width page nfree room stream"
PLAN_OK = dict(lens=A, new=A + 0x100, table=A + 0x1000, free=A + 0x200, count=A + 0x300, cq=A + 0x400, out=A + 0x500,
               slots=A + 0x2000, left=A + 0x600, b=4, width=8, page=16, nfree=9, room=50, stream=None)


@pytest.mark.parametrize("kw,expect", [
    (dict(lens=None), INV), (dict(free=None), INV), (dict(left=None), INV), (dict(slots=A + 0x2004), INV),
    (dict(count=A + 0x301), INV), (dict(b=0), INV), (dict(width=0), INV), (dict(page=0), INV), (dict(nfree=0), INV),
    (dict(room=0), INV), (dict(b=70000), UNS), (dict(width=1 << 20, page=1 << 12), UNS),
    # outputs over inputs, and over each other
    (dict(out=A), INV), (dict(left=A + 0x300), INV), (dict(cq=A + 0x10c), INV), (dict(table=A + 0x1f0), INV),
    (dict(out=A + 0x40c), INV), (dict(slots=A + 0x1000), INV),
])
def test_paged_plan_refuses(exattn_lib, kw, expect):
    assert call(exattn_lib.attn_paged_plan, PLAN, **{**PLAN_OK, **kw}) == expect


WRITE = "k v slots kp vp t hk d pages page ks vs dtype stream"
WRITE_OK = dict(k=A, v=A, slots=A, kp=A, vp=A, t=5, hk=2, d=64, pages=3, page=16, ks=128, vs=128,
                dtype=ea.ATTN_FP16, stream=None)


@pytest.mark.parametrize("kw,expect", [
    (dict(k=None), INV), (dict(slots=None), INV), (dict(vp=A + 4), INV), (dict(slots=A + 4), INV), (dict(t=0), INV),
    (dict(hk=0), INV), (dict(page=0), INV), (dict(pages=0), INV), (dict(ks=120), INV), (dict(vs=130), INV),
    (dict(dtype=3), INV), (dict(d=20), UNS), (dict(hk=70000, ks=1 << 24, vs=1 << 24), UNS),
])
def test_paged_write_refuses(exattn_lib, kw, expect):
    assert call(exattn_lib.attn_paged_write, WRITE, **{**WRITE_OK, **kw}) == expect


def test_binding_refuses_host_tensors():
    q = torch.zeros(4, 2, 64, dtype=torch.float16)
    cu = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ea.attn_fwd_packed(q, q, q, cu, cu)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ea.attn_bwd_packed(q, q, q, q, q, q, cu, cu)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ea.attn_chunk_paged(q, q, q, cu, cu, cu)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ea.attn_paged_plan(cu, cu, cu, cu, cu, 16, max_tokens=4)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ea.attn_paged_write(q, q, cu, q, q)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ea.attn_fwd_packed(None, q, q, cu, cu)


# ---------------------------------------------------------------- the oracle's own pins
@pytest.mark.parametrize("causal", [False, True])
def test_packed_oracle_by_hand(oracle_mod, causal):
    """Each row by the definition, with loops."""
    g = np.random.default_rng(3)
    cq, ck = [0, 3, 3, 5], [0, 2, 4, 10]
    q, k, v = g.standard_normal((5, 4, 8)), g.standard_normal((10, 2, 8)), g.standard_normal((10, 2, 8))
    o, lse = oracle_mod.packed_attention(q, k, v, cq, ck, 0.3, causal)
    for i in range(3):
        sq, sk = cq[i + 1] - cq[i], ck[i + 1] - ck[i]
        for r in range(sq):
            for h in range(4):
                keys = [j for j in range(sk) if not causal or j <= r + sk - sq]
                s = [0.3 * float(q[cq[i] + r, h] @ k[ck[i] + j, h // 2]) for j in keys]
                z = sum(np.exp(s))
                want = sum((np.exp(x) / z * v[ck[i] + j, h // 2] for x, j in zip(s, keys)), np.zeros(8))
                assert np.allclose(o[cq[i] + r, h], want, atol=1e-13)
                assert (not keys and np.isneginf(lse[h, cq[i] + r])) or np.isclose(lse[h, cq[i] + r], np.log(z))


@pytest.mark.parametrize("causal", [False, True])
def test_packed_oracle_gradients_by_differences(oracle_mod, causal):
    """The chain rule with grouped heads against central differences of a scalar of the outputs."""
    g = np.random.default_rng(4)
    cq, ck = [0, 3, 4, 7], [0, 4, 4, 6]
    x = [g.standard_normal((7, 4, 8)), g.standard_normal((6, 2, 8)), g.standard_normal((6, 2, 8))]
    w = g.standard_normal((7, 4, 8))
    grads = oracle_mod.packed_attention_backward(*x, w, cq, ck, 0.4, causal)

    def value():
        return float((oracle_mod.packed_attention(*x, cq, ck, 0.4, causal)[0] * w).sum())

    step = 1e-5
    for a, grad in zip(x, grads):
        for at in [tuple(g.integers(0, n) for n in a.shape) for _ in range(25)]:
            keep = a[at]
            a[at] = keep + step
            up = value()
            a[at] = keep - step
            down = value()
            a[at] = keep
            assert abs((up - down) / (2 * step) - grad[at]) < 1e-7


def test_plan_oracle_by_hand(oracle_mod):
    """Pages of 4: request 0 has 3 keys and brings 2, request 1 none and 5, request 2 brings nothing."""
    table, cu, lens, slots, left = oracle_mod.paged_plan(
        np.array([3, 0, 8]), np.array([2, 5, 0]), np.array([[7, -1, -1], [-1, -1, -1], [1, 2, -1]]),
        np.array([9, 8, 6, 5]), 4, 4, 9)
    assert table.tolist() == [[7, 5, -1], [6, 8, -1], [1, 2, -1]]
    assert cu.tolist() == [0, 2, 7, 7] and lens.tolist() == [5, 5, 8] and left == 1
    assert slots.tolist() == [7 * 4 + 3, 5 * 4, 24, 25, 26, 27, 32, -1, -1]
