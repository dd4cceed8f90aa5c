"""Groups of small values going into a 4-bit cache, whose scales are subnormal
e4m3 numbers (k 2^-9, k < 8) or just above: a group's largest magnitude lies on the
border between two scales, or is a neighbour of one in its type, so that a
quotient by the scale reaches almost 9 (k = 1) and is limited to 6.

The bits are the oracle's: with a power of two as the tensor's scale, borders of
scales are exact in fp32 and their neighbours in a 16-bit type are 2^-12 of their
size away, as are borders of codes (x is a multiple of the scale's step there).
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def groups(dtype, tensor_scale):
    """[n, 1, 32]: n rows of two groups, the second in reverse."""
    rows = []
    codes = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    for k in range(10):
        m = torch.tensor(6.0 * (k + 0.5) * 2.0 ** -9 * tensor_scale, dtype=dtype)
        assert m.double().item() == 6.0 * (k + 0.5) * 2.0 ** -9 * tensor_scale
        up, down = (torch.nextafter(m, torch.tensor(x, dtype=dtype)) for x in (float("inf"), 0.0))
        for top in (m, up, down):
            # borders between codes at either of the two scales that m may get
            x = [top] + [c * s * 2.0 ** -9 * tensor_scale for s in (k, k + 1) for c in codes] + [-top]
            x = torch.stack([torch.as_tensor(v).to(dtype).clamp(-top, top) for v in x])
            x[2::3] = -x[2::3]
            rows.append(torch.cat([x, x.flip(0)]))
    return torch.stack(rows)[:, None]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("tensor_scale", [1.0, 0.25, 16.0])
def test_subnormal_scales(gpu, oracle_mod, dtype, tensor_scale):
    x = groups(dtype, tensor_scale)
    n, page = x.shape[0], 16
    want_code, want_s = oracle_mod.q4_quantise(x, tensor_scale)
    assert {0, 1, 2, 4, 7, 8} <= set(want_s.ravel().tolist())
    unit = np.repeat(oracle_mod.E4M3[want_s] * tensor_scale, 16, -1)
    y = np.abs(x.double().numpy()) / np.where(unit > 0, unit, np.inf)
    assert 8.9 < y.max() < 9
    pages = -(-n // page)
    kp, vp = (torch.zeros((pages, 1, gpu.attn_q4_page_bytes(page, 32)), dtype=torch.uint8, device="cuda") for _ in "kv")
    cs = torch.tensor([[1.0] * 16 + [0.0] * 16], device="cuda")  # (turns nothing)
    at = torch.arange(n, device="cuda")
    v = x.cuda()
    gpu.attn_paged_append_q4(v, v, v, cs, torch.zeros_like(at), at, kp, vp, k_scale=tensor_scale, v_scale=tensor_scale)
    for pool in (kp, vp):
        code, s = (r[:n] for r in oracle_mod.q4_rows(pool.cpu().numpy(), 32))
        assert np.array_equal(s, want_s)
        assert np.all((code == want_code) | ((code | want_code) == 8)), "codes (0 has two)"
