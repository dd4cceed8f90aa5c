"""Workspaces belong to a stream, not to its handle: a stream destroyed with a
call still to do, and a new one that CUDA may give the same handle, at work at
the same time. Whether the handle comes back is CUDA's choice; the results
have to be right either way.
"""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu


class Raw:
    """A stream of the CUDA runtime's own, destroyed when told to."""

    def __init__(self):
        self.handle = ctypes.c_void_p()
        at = ctypes.addressof(self.handle)
        assert int(torch.cuda.cudart().cudaStreamCreate(at)) == 0
        self.stream = torch.cuda.ExternalStream(self.handle.value)

    def destroy(self):
        assert int(torch.cuda.cudart().cudaStreamDestroy(self.handle.value)) == 0


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def packed(gpu, keys, seed):
    """One row over many keys: cut units, joined through the workspace."""
    torch.manual_seed(seed)
    q = torch.randn(1, 4, 128, device="cuda", dtype=torch.bfloat16)
    k, v = (torch.randn(keys, 1, 128, device="cuda", dtype=torch.bfloat16) for _ in "kv")
    cq, ck = ints([0, 1]), ints([0, keys])
    out, lse = torch.empty_like(q), torch.empty(4, 1, device="cuda")
    return lambda s: gpu.attn_fwd_packed(q, k, v, cq, ck, out=out, lse=lse, stream=s)


def decode(gpu, keys, seed):
    torch.manual_seed(seed)
    q = torch.randn(1, 1, 2, 128, device="cuda", dtype=torch.bfloat16)
    k, v = (torch.randn(1, keys, 2, 128, device="cuda", dtype=torch.bfloat16) for _ in "kv")
    out, lse = torch.empty_like(q), torch.empty(1, 2, 1, device="cuda")
    return lambda s: gpu.attn_decode_splitkv(q, k, v, out=out, lse=lse, num_splits=12, stream=s)


def same(got, want, exact):
    if exact:
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        return
    # the split decode's two reduces add up the same partials in fp32 and round
    # O once each: half a step of bf16 on either side; LSE near 10
    (o, lse), (o2, lse2) = got, want
    assert torch.all((o.float() - o2.float()).abs() <= 2 ** -7 * o2.float().abs() + 2 ** -20)
    assert torch.all((lse - lse2).abs() <= 2 ** -18)


@pytest.mark.parametrize("make,exact", [(packed, True), (decode, False)])
def test_a_destroyed_stream_and_its_successor(gpu, make, exact):
    first, second = make(gpu, 20000, 1), make(gpu, 33000, 2)
    want = [[x.clone() for x in f(None)] for f in (first, second)]
    torch.cuda.synchronize()
    again = 0
    for _ in range(12):
        a = Raw()
        got = first(a.stream)                # the stream's workspace is made
        a.stream.synchronize()
        for x in got:
            x.fill_(7.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(a.stream):
            torch.cuda._sleep(20_000_000)    # some 10 ms
        got = first(a.stream)                # still to do when the stream goes
        a.destroy()
        b = Raw()
        again += b.handle.value == a.handle.value
        other = second(b.stream)             # a larger workspace: the smaller one's place is given up
        third = second(b.stream)
        torch.cuda.synchronize()
        b.destroy()
        assert gpu.attn_get_device_status() == gpu.ATTN_OK
        same(got, want[0], exact)
        same(other, want[1], exact)
        same(third, want[1], exact)
    print("handles that came back:", again, "of 12")
