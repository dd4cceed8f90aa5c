"""Refusals of the rotating appends and of the 4-bit cache's entry points, and
pins of their oracle; no GPU. (Addresses are never dereferenced.)
"""
import numpy as np
import pytest
import torch

import exact_attention_65_gb300 as ea

A = 0x10000
INV, UNS = ea.ATTN_ERR_INVALID_ARG, ea.ATTN_ERR_UNSUPPORTED

APPEND = "q k v cs pos slots out kp vp t far rot pairs h hk d pages page qs ks vs os dtype stream"
APPEND_OK = dict(q=A, k=A, v=A, cs=A, pos=A, slots=A, out=A, kp=A, vp=A, t=5, far=9, rot=64, pairs=0, h=4, hk=2, d=64,
                 pages=3, page=16, qs=256, ks=128, vs=128, os=256, dtype=ea.ATTN_BF16, stream=None)
APPEND_Q4 = APPEND.replace("os dtype", "os k_scale v_scale dtype")
APPEND_Q4_OK = dict(APPEND_OK, k_scale=1.0, v_scale=1.0)


def call(fn, order, **kw):
    return fn(*[kw[x] for x in order.split()])


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), INV), (dict(k=None), INV), (dict(cs=None), INV), (dict(pos=None), INV), (dict(slots=None), INV),
    (dict(out=None), INV), (dict(vp=None), INV), (dict(v=A + 8), INV), (dict(cs=A + 4), INV), (dict(pos=A + 4), INV),
    (dict(out=A + 2), INV), (dict(kp=A + 8), INV), (dict(t=0), INV), (dict(far=0), INV), (dict(h=0), INV),
    (dict(hk=0), INV), (dict(pages=0), INV), (dict(page=0), INV), (dict(dtype=5), INV), (dict(qs=248), INV),
    (dict(os=200), INV), (dict(ks=129), INV), (dict(vs=64), INV), (dict(d=48), UNS), (dict(rot=0), UNS),
    (dict(rot=24), UNS), (dict(rot=80), UNS), (dict(h=70000, qs=1 << 24, os=1 << 24), UNS), (dict(far=1 << 31), UNS),
    (dict(t=1 << 31), UNS),
])
def test_appends_refuse(exattn_lib, kw, expect):
    assert call(exattn_lib.attn_paged_append, APPEND, **{**APPEND_OK, **kw}) == expect
    assert call(exattn_lib.attn_paged_append_q4, APPEND_Q4, **{**APPEND_Q4_OK, **kw}) == expect


SCALES = [(dict(k_scale=0.0), INV), (dict(v_scale=-1.0), INV), (dict(k_scale=float("nan")), INV),
          (dict(v_scale=float("inf")), INV), (dict(k_scale=1e-30), INV), (dict(v_scale=1e30), INV),
          (dict(page=24), UNS), (dict(page=8), UNS)]


@pytest.mark.parametrize("kw,expect", SCALES)
def test_append_q4_refuses(exattn_lib, kw, expect):
    assert call(exattn_lib.attn_paged_append_q4, APPEND_Q4, **{**APPEND_Q4_OK, **kw}) == expect


READ = "kp vp slots k v t hk d pages page k_scale v_scale ks vs dtype stream"
READ_OK = dict(kp=A, vp=A, slots=A, k=A, v=A, t=5, hk=2, d=64, pages=3, page=16, k_scale=1.0, v_scale=1.0, ks=128,
               vs=128, dtype=ea.ATTN_FP16, stream=None)


@pytest.mark.parametrize("kw,expect", SCALES + [
    (dict(kp=None), INV), (dict(slots=None), INV), (dict(k=None), INV), (dict(vp=A + 8), INV), (dict(v=A + 8), INV),
    (dict(slots=A + 4), INV), (dict(t=0), INV), (dict(hk=0), INV), (dict(pages=0), INV), (dict(page=0), INV),
    (dict(dtype=2), INV), (dict(ks=120), INV), (dict(vs=0), INV), (dict(d=8), UNS),
    (dict(hk=70000, ks=1 << 24, vs=1 << 24), UNS), (dict(t=1 << 31), UNS),
])
def test_read_q4_refuses(exattn_lib, kw, expect):
    assert call(exattn_lib.attn_paged_read_q4, READ, **{**READ_OK, **kw}) == expect


CHUNK = "q kp vp table cq lens o lse b tq mq h hk d pages page width qs scale k_scale v_scale causal dtype stream"
CHUNK_OK = dict(q=A, kp=A, vp=A, table=A, cq=A, lens=A, o=A, lse=A, b=2, tq=10, mq=0, h=4, hk=2, d=64, pages=9, page=16,
                width=4, qs=256, scale=0.1, k_scale=1.0, v_scale=1.0, causal=1, dtype=ea.ATTN_BF16, stream=None)


@pytest.mark.parametrize("kw,expect", SCALES + [
    (dict(q=None), INV), (dict(kp=None), INV), (dict(table=None), INV), (dict(lens=None), INV), (dict(lse=None), INV),
    (dict(vp=A + 8), INV), (dict(o=A + 8), INV), (dict(table=A + 2), INV), (dict(cq=A + 1), INV), (dict(b=0), INV),
    (dict(tq=0), INV), (dict(pages=0), INV), (dict(page=0), INV), (dict(width=0), INV), (dict(h=6, hk=4), INV),
    (dict(qs=64), INV), (dict(dtype=2), INV), (dict(scale=float("inf")), INV), (dict(scale=1e38, k_scale=1e10), INV),
    (dict(d=96), UNS), (dict(h=258, hk=2, qs=1 << 15), UNS), (dict(page=1 << 20, width=1 << 12), UNS),
    (dict(tq=0x7fffffff), UNS), (dict(b=70000), UNS),
])
def test_chunk_q4_refuses(exattn_lib, kw, expect):
    assert call(exattn_lib.attn_chunk_paged_q4, CHUNK, **{**CHUNK_OK, **kw}) == expect


def test_page_bytes(exattn_lib):
    assert [ea.attn_q4_page_bytes(16, d) for d in (16, 32, 64, 128)] == [144, 288, 576, 1152]
    assert ea.attn_q4_page_bytes(48, 128) == 3456
    assert [ea.attn_q4_page_bytes(*x) for x in ((0, 64), (8, 64), (24, 64), (16, 48), (-16, 64))] == [0] * 5


def test_binding_refuses_host_tensors(exattn_lib):
    q = torch.zeros(4, 2, 64, dtype=torch.float16)
    n = torch.zeros(4, dtype=torch.int64)
    for fn in (ea.attn_paged_append, ea.attn_paged_append_q4):
        with pytest.raises(ValueError, match="CUDA tensor"):
            fn(q, q, q, torch.zeros(9, 64), n, n, q, q)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ea.attn_paged_read_q4(q, q, n, 64)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ea.attn_chunk_paged_q4(q, q, q, n, n, n)


# ---------------------------------------------------------------- the oracle's own pins
def test_rotation_by_hand(oracle_mod):
    """A quarter turn takes (a, b) to (-b, a); the channels behind pass."""
    x = np.arange(1.0, 9.0).reshape(1, 1, 8)
    cs = np.array([[1.0, 1.0, 0.0, 0.0], [0.0, 1.0, 1.0, 0.0]])  # pair 0 turns at position 1
    assert oracle_mod.rotate(x, cs, [0])[0, 0].tolist() == x[0, 0].tolist()
    assert oracle_mod.rotate(x, cs, [1])[0, 0].tolist() == [-3, 2, 1, 4, 5, 6, 7, 8]
    assert oracle_mod.rotate(x, cs, [1], True)[0, 0].tolist() == [-2, 1, 3, 4, 5, 6, 7, 8]


def test_formats_by_hand(oracle_mod):
    """Every e4m3 value against torch's type; ties and ends of both grids."""
    t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn)
    assert np.array_equal(oracle_mod.E4M3, t.double().numpy())
    assert oracle_mod.nearest(oracle_mod.E2M1, np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 9.0])).tolist() == \
        [0, 2, 2, 4, 4, 6, 6, 7]
    assert oracle_mod.nearest(oracle_mod.E4M3, np.array([1.0625, 1.1875, 2.0 ** -10, 500.0])).tolist() == [56, 58, 0, 126]
    x = np.random.default_rng(1).standard_normal((5, 2, 32)) * 3
    code, s = oracle_mod.q4_quantise(x, 0.5)
    back = oracle_mod.q4_values(code, s, 0.5)
    m = np.abs(x.reshape(5, 2, 2, 16)).max(-1, keepdims=True)
    # half a step of the widest kind (4 to 6), and the scale's own rounding
    assert np.all(np.abs(back - x).reshape(m.shape[:-1] + (16,)) <= m / 6 * (1 + 1 / 16) * 1.0 + 6 / 16 * m / 6 + 1e-12)
    pool = oracle_mod.q4_pool(*(np.concatenate([y, y[:1].repeat(11, 0)]) for y in (code, s)), 1, 16)
    code2, s2 = oracle_mod.q4_rows(pool, 32)
    assert np.array_equal(code2[:5], code) and np.array_equal(s2[:5], s)
    # channel 0 in the low half of byte 0, the scales behind 16 rows of codes
    assert pool.shape == (1, 2, 16 * 18) and pool[0, 0, 0] == code[0, 0, 0] | code[0, 0, 1] << 4
    assert pool[0, 1, 16 * 16] == s[0, 1, 0]
