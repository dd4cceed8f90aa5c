"""Units that see no key, several in a row on one CTA: causal rows before the
first key, requests without keys, key ranges past the end. Such a unit makes
no product, so nothing but the hand-back of its accumulators keeps the issuer
from running two phases of a barrier ahead of the epilogue, which would then
wait for a phase that is past. O = 0 and LSE = -inf there, and the other rows
as ever.
"""
import math

import numpy as np
import pytest
import torch

import workloads
from parity import compare, compare_masked

pytestmark = pytest.mark.gpu


def check_forward(ea, oracle_mod, o, lse, q, k, v):
    """Rows that see no key, and a sample of the others against the oracle."""
    assert ea.attn_get_device_status() == ea.ATTN_OK
    sq, sk = q.shape[1], k.shape[1]
    hidden = max(sq - sk, 0)
    assert torch.all(o[:, :hidden] == 0) and torch.all(torch.isneginf(lse[:, :, :hidden]))
    rows = sorted({max(hidden - 1, 0), hidden, hidden + 1, sq - 1} & set(range(sq)))
    o_ref, lse_ref = oracle_mod.attention(q, k, v, 1 / math.sqrt(q.shape[3]), rows=rows, causal=True)
    compare_masked(o, lse, o_ref, lse_ref, rows=rows)


@pytest.mark.parametrize("b,sq,sk,h", [
    (2, 1024, 10, 76),    # four units a head, three of them without keys: every SM has several
    (1, 2000, 200, 100),
    (1, 5000, 1, 60),
])
@pytest.mark.parametrize("d", [16, 128])
def test_forward_with_many_more_rows_than_keys(gpu, oracle_mod, b, sq, sk, h, d):
    q, k, v = workloads.make_qkv(b, sq, sk, h, d, torch.bfloat16, seed=101)
    o, lse = gpu.attn_fwd(*(t.cuda() for t in (q, k, v)), causal=True)
    check_forward(gpu, oracle_mod, o, lse, q, k, v)


@pytest.mark.parametrize("sq", [5, 300])
def test_paged_requests_without_keys(gpu, oracle_mod, sq):
    """Several new rows each for 400 requests, most of them without a key (the
    one-tile kernel, and the two-tile one)."""
    b, h, d, page, width = 400, 2, 64, 16, 12
    r = np.random.default_rng(7)
    lens = np.where(r.random(b) < 0.9, 0, r.integers(1, page * width + 1, b))
    lens[-1] = page * width
    kp, vp = (torch.randn(b * width, page, h, d, generator=torch.Generator().manual_seed(i)).bfloat16() for i in (1, 2))
    table = torch.arange(b * width, dtype=torch.int32).view(b, width)
    q = torch.randn(b, sq, h, d, generator=torch.Generator().manual_seed(3)).bfloat16()
    o, lse = gpu.attn_decode_paged(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(),
                                   torch.tensor(lens, dtype=torch.int32).cuda(), num_splits=1)
    assert gpu.attn_get_device_status() == gpu.ATTN_OK
    none = torch.tensor(lens == 0).cuda()
    assert torch.all(o[none] == 0) and torch.all(torch.isneginf(lse[none]))
    rows = sorted({0, sq - 1})
    for i in np.flatnonzero(lens)[-6:]:
        keys, values = (x.view(b, width * page, h, d)[i:i + 1, :lens[i]] for x in (kp, vp))
        o_ref, lse_ref = oracle_mod.attention(q[i:i + 1], keys.contiguous(), values.contiguous(), 0.125, rows=rows)
        compare(o[i:i + 1], lse[i:i + 1], o_ref, lse_ref, rows=rows)


def test_key_ranges_past_the_end(gpu, oracle_mod):
    """Most requests end in the first of many key ranges."""
    b, sq, h, d, page, width = 40, 4, 2, 128, 16, 64
    lens = [1 if i % 8 else page * width for i in range(b)]
    kp, vp = (torch.randn(b * width, page, h, d, generator=torch.Generator().manual_seed(i)).bfloat16() for i in (4, 5))
    table = torch.arange(b * width, dtype=torch.int32).view(b, width)
    q = torch.randn(b, sq, h, d, generator=torch.Generator().manual_seed(6)).bfloat16()
    for causal in (False, True):
        o, lse = gpu.attn_decode_paged(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(),
                                       torch.tensor(lens, dtype=torch.int32).cuda(), num_splits=8, causal=causal)
        assert gpu.attn_get_device_status() == gpu.ATTN_OK
        for i in (0, 1, 8, 39):
            keys, values = (x.view(b, width * page, h, d)[i:i + 1, :lens[i]].contiguous() for x in (kp, vp))
            o_ref, lse_ref = oracle_mod.attention(q[i:i + 1], keys, values, 1 / math.sqrt(d), rows=list(range(sq)),
                                                  causal=causal)
            compare_masked(o[i:i + 1], lse[i:i + 1], o_ref, lse_ref, rows=list(range(sq)))


@pytest.mark.parametrize("b,sq,sk,h", [
    (2, 1024, 10, 60),   # seven of eight query tiles see no key
    (1, 10, 3000, 60),   # all keys are seen
    (1, 2000, 200, 60),
])
def test_backward_with_many_more_rows_than_keys(gpu, oracle_mod, b, sq, sk, h):
    """dQ = 0 in the rows that see no key; the gradients of two heads against the oracle."""
    d = 128
    q, k, v = workloads.make_qkv(b, sq, sk, h, d, torch.bfloat16, seed=103)
    g = torch.randn(q.shape, generator=torch.Generator().manual_seed(104)).bfloat16()
    dev = [t.cuda() for t in (q, k, v)]
    o, lse = gpu.attn_fwd(*dev, causal=True)
    grads = gpu.attn_bwd(*dev, o, lse, g.cuda(), causal=True)
    assert gpu.attn_get_device_status() == gpu.ATTN_OK
    assert torch.all(grads[0][:, :max(sq - sk, 0)] == 0)
    for head in (0, h - 1):
        part = [x[:, :, head:head + 1].contiguous() for x in (q, k, v, g)]
        refs = oracle_mod.attention_backward(*part, 1 / math.sqrt(d), causal=True)
        for x, ref in zip(grads, refs):
            got = x[:, :, head:head + 1].double().cpu().numpy()
            assert np.isfinite(got).all()
            assert np.abs(got - ref).max() <= 2e-2 * (1 + np.abs(ref).max())
