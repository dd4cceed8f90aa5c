"""More than 32 sequences with cut units: the place of a CTA's share is then
looked for 32 sequences at a time, with what lies before carried on, and the
line's sums come from the whole block. Short and empty sequences with long
ones behind the 32nd and at the end, every result checked.
"""
import numpy as np
import pytest
import torch

import test_chunk_paged_gpu as chunk
import test_packed_bwd_gpu as backward
import test_packed_gpu as forward
from test_packed_plan import plan

pytestmark = pytest.mark.gpu


def batch(count, long, seed):
    """Rows and keys of `count` sequences, those of `long` ({index: (rows, keys)}) given."""
    r = np.random.default_rng(seed)
    rows = [int(r.choice([0, 1, 1, 2, 5])) for _ in range(count)]
    keys = [n + int(r.choice([0, 0, 7, 40])) for n in rows]
    for i, (n, m) in long.items():
        rows[i % count], keys[i % count] = n, m
    return rows, keys


def cut_behind_the_32nd(lib, rows, keys, h, h_kv, one_tile, causal, by_key):
    return any(r["slot"] >= 0 and r["seq"] >= 32 for r in plan(lib, rows, keys, h, h_kv, one_tile, causal, by_key))


LONG = {
    "late": {33: (3, 7000)},
    "last": {-1: (20, 9000)},
    "both": {40: (9, 5000), -1: (1, 12000)},
    "each side": {3: (30, 6000), 35: (17, 4000), 64: (2, 8000)},
}


@pytest.mark.parametrize("where", sorted(LONG))
@pytest.mark.parametrize("causal", [False, True])
def test_forward_one_tile(gpu, exattn_lib, oracle_mod, where, causal):
    rows, keys = batch(70, LONG[where], 1)
    assert cut_behind_the_32nd(exattn_lib, rows, keys, 4, 1, 1, causal, 0)
    forward.run(gpu, oracle_mod, rows, keys, 4, 1, 64, torch.bfloat16, causal)
    forward.run(gpu, oracle_mod, rows, keys, 4, 1, 16, torch.float16, causal, tail=5)


@pytest.mark.parametrize("long", [{45: (700, 6000)}, {-1: (900, 5000)}, {34: (600, 4000), -1: (300, 9000)}])
@pytest.mark.parametrize("causal", [False, True])
def test_forward_two_tiles(gpu, exattn_lib, oracle_mod, long, causal):
    rows, keys = batch(49, long, 2)
    assert cut_behind_the_32nd(exattn_lib, rows, keys, 2, 1, 0, causal, 0)
    forward.run(gpu, oracle_mod, rows, keys, 2, 1, 128, torch.bfloat16, causal, tail=3)


@pytest.mark.parametrize("where", sorted(LONG))
@pytest.mark.parametrize("hint", [False, True])
def test_chunks(gpu, oracle_mod, where, hint):
    rows, keys = batch(70, LONG[where], 3)
    chunk.run(gpu, oracle_mod, rows, keys, 4, 1, 64, 16, torch.bfloat16, hint=hint)


@pytest.mark.parametrize("long", [{33: (40, 6000)}, {-1: (1500, 1500)}, {3: (30, 3000), 41: (1100, 1100), -1: (5, 5000)}])
@pytest.mark.parametrize("causal", [False, True])
def test_backward(gpu, exattn_lib, oracle_mod, long, causal):
    rows, keys = batch(53, long, 4)
    assert cut_behind_the_32nd(exattn_lib, rows, keys, 4, 1, 1, causal, 0) or \
        cut_behind_the_32nd(exattn_lib, rows, keys, 4, 1, 1, causal, 1)
    backward.run(gpu, oracle_mod, rows, keys, 4, 1, 64, torch.bfloat16, causal, tail=4)
    backward.run(gpu, oracle_mod, rows, keys, 4, 1, 32, torch.float16, causal, fused=True)
