"""Calls of several host threads at once: on a stream each, and on one stream,
whose workspace they then share. (The binding releases the interpreter's lock
inside a call.) Each thread's results are those it gets alone.
"""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def rows(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


def packed(ea, i):
    """Cut units, another number of them for each thread; forward and backward."""
    n, m = 2 + i, 4000 + 3000 * i
    q, k, v, g = (rows(10 * i + j, x, y, 64) for j, (x, y) in enumerate(((n, 4), (m, 2), (m, 2), (n, 4))))
    cq, ck = ints([0, n]), ints([0, m])
    o, lse = torch.empty_like(q), torch.empty(4, n, device="cuda")
    grads = [torch.empty_like(x) for x in (q, k, v)]

    def call(s):
        ea.attn_fwd_packed(q, k, v, cq, ck, out=o, lse=lse, causal=True, stream=s)
        ea.attn_bwd_packed(q, k, v, o, lse, g, cq, ck, dq=grads[0], dk=grads[1], dv=grads[2], causal=True, stream=s)

    return call, [o, lse, *grads]


def decode(ea, i):
    """Key ranges with a reduce, in one kernel (one row) or a second one (several)."""
    sq, sk = (1, 6000 + 5000 * i) if i % 2 == 0 else (4 + i, 5000 * i)
    q, k, v = (rows(100 + 10 * i + j, 1, n, 3, 64) for j, n in enumerate((sq, sk, sk)))
    o, lse = torch.empty_like(q), torch.empty(1, 3, sq, device="cuda")
    return lambda s: ea.attn_decode_splitkv(q, k, v, out=o, lse=lse, num_splits=4 + 3 * i, stream=s), [o, lse]


@pytest.mark.parametrize("one_stream", [False, True])
@pytest.mark.parametrize("make", [packed, decode])
def test_threads(gpu, make, one_stream):
    count = 4
    jobs = [make(gpu, i) for i in range(count)]
    want = []
    for call, outs in jobs:
        call(None)
        want.append([x.clone() for x in outs])
    shared = torch.cuda.Stream()
    streams = [shared if one_stream else torch.cuda.Stream() for _ in range(count)]
    torch.cuda.synchronize()
    wrong, go = [], threading.Barrier(count)

    def work(i):
        try:
            call, outs = jobs[i]
            torch.cuda.set_device(0)
            for _ in range(15):
                go.wait(60)
                with torch.cuda.stream(streams[i]):
                    for x in outs:
                        x.fill_(7.0)
                for _ in range(5):
                    call(streams[i])
                streams[i].synchronize()
                if not all(torch.equal(x, y) for x, y in zip(outs, want[i])):
                    wrong.append(i)
        except Exception as e:  # noqa: BLE001 (reported by the test)
            wrong.append(repr(e))
            go.abort()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(count)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert gpu.attn_get_device_status() == gpu.ATTN_OK
    assert wrong == []
