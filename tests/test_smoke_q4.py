"""The smoke run of the 4-bit cache notices a mistake in any of its three results.
The library is stood in for by the oracle here, on the CPU; the mistakes are in
the oracle that the smoke run compares with.
"""
import numpy as np
import pytest
import torch

import __graft_entry__ as entry


class Library:
    """The entry points that smoke_q4() calls, from the oracle."""
    ATTN_OK = 0

    def __init__(self, oracle):
        self.oracle = oracle

    def attn_get_device_status(self):
        return self.ATTN_OK

    def attn_q4_page_bytes(self, page, d):
        return page * 9 * d // 16

    def attn_paged_plan(self, lens, new, table, free, count, page, max_tokens):
        got = self.oracle.paged_plan(lens.tolist(), new.tolist(), table.numpy(), free.tolist(), count.tolist()[0], page,
                                     max_tokens)
        table.copy_(torch.tensor(np.asarray(got[0])))
        return [torch.tensor(np.asarray(x)) for x in got[1:]]

    def rotated(self, x, cs, pos):
        return torch.tensor(self.oracle.rotate(x, cs, pos)).to(x.dtype)

    def attn_paged_append(self, q, k, v, cs, pos, slots, k_pages, v_pages):
        k_pages.flatten(0, 1)[slots], v_pages.flatten(0, 1)[slots] = self.rotated(k, cs, pos), v
        return self.rotated(q, cs, pos)

    def attn_paged_append_q4(self, q, k, v, cs, pos, slots, k_pages, v_pages):
        n, _, block = k_pages.shape
        d = q.shape[2]
        page = block * 16 // (9 * d)
        for pool, x in ((k_pages, self.oracle.rotate(k, cs, pos)), (v_pages, v)):
            code, s = self.oracle.q4_rows(pool.numpy(), d)
            code[slots.numpy()], s[slots.numpy()] = self.oracle.q4_quantise(x, 1.0)
            pool.copy_(torch.tensor(self.oracle.q4_pool(code, s, n, page)))
        return self.rotated(q, cs, pos)

    def attn_paged_read_q4(self, k_pages, v_pages, slots, d):
        return [torch.tensor(self.oracle.q4_values(*(x[slots.numpy()] for x in self.oracle.q4_rows(p.numpy(), d)), 1.0))
                .to(torch.bfloat16) for p in (k_pages, v_pages)]

    def attn_chunk_paged_q4(self, q, k_pages, v_pages, table, cu, lens, max_seqlen_q, causal):
        d, block = q.shape[2], k_pages.shape[2]
        page = block * 16 // (9 * d)
        at = np.concatenate([t[np.arange(n) // page] * page + np.arange(n) % page
                             for t, n in zip(table.numpy(), lens.tolist())])
        k, v = (self.oracle.q4_values(*(x[at] for x in self.oracle.q4_rows(p.numpy(), d)), 1.0)
                for p in (k_pages, v_pages))
        o, lse = self.oracle.packed_attention(q, k, v, cu.numpy(), np.concatenate([[0], np.cumsum(lens.numpy())]),
                                              d ** -0.5, causal=causal)
        return torch.tensor(o).to(q.dtype), torch.tensor(lse).float()


class Wrong:
    """The oracle with a mistake in one result."""

    def __init__(self, oracle, which):
        self.oracle, self.which = oracle, which

    def rotate(self, *args):
        x = self.oracle.rotate(*args)
        return x * (1 + 2.0 ** -6) if self.which == "keys" else x

    def packed_attention(self, *args, **kw):
        o, lse = self.oracle.packed_attention(*args, **kw)
        return o + 0.04 * (self.which == "O"), lse + 0.05 * (self.which == "LSE")


def test_smoke_passes(oracle_mod):
    assert entry.smoke_q4(Library(oracle_mod), Wrong(oracle_mod, "nothing"), "cpu") <= 2e-2


@pytest.mark.parametrize("which,says", [("keys", "rotated keys"), ("O", "4-bit cache"), ("LSE", "4-bit cache")])
def test_smoke_notices(oracle_mod, which, says):
    with pytest.raises(RuntimeError, match=says):
        entry.smoke_q4(Library(oracle_mod), Wrong(oracle_mod, which), "cpu")
