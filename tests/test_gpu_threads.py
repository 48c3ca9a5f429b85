"""Threads that call one layer on one stream, each with inputs of its own, get what one thread gets."""
import threading

import pytest
import torch

from test_gpu_block_cache import _attend
from test_gpu_w4 import _make

pytestmark = pytest.mark.gpu


def _together(works, repeat=60):
    """Each of `works` in a thread of its own, on the current stream; their last results."""
    out, failed, go = [None] * len(works), [], threading.Barrier(len(works))

    def body(i):
        try:
            go.wait()
            for _ in range(repeat):
                out[i] = works[i]()
        except Exception as e:        # seen below, in the test's own thread
            failed.append(e)
    threads = [threading.Thread(target=body, args=(i,)) for i in range(len(works))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    return out


@pytest.mark.parametrize("T", [(6, 6), (40, 40), (300, 300), (3, 300), (300, 20)])
def test_gate_out_w4(T):
    model, w4, g = _make(1024, 16, 64, gate="channel")
    o = [torch.randn(t, 2048, generator=g, device="cuda").bfloat16() for t in T]
    z = [torch.randn(t, 2048, generator=g, device="cuda") for t in T]
    want = [model.gate_out_w4(a, w4, b) for a, b in zip(o, z)]
    torch.cuda.synchronize()
    got = _together([lambda a=a, b=b: model.gate_out_w4(a, w4, b) for a, b in zip(o, z)])
    model.sync_status()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("H", [16, 32])
def test_block_scaled_decode(H):
    model, pool, q, z, L, o = _attend(H, [1500, 130, 900, 333], 64, 32, seed=31)
    q2, few = q.flip(0).contiguous(), torch.tensor([3], dtype=torch.int32, device="cuda")
    calls = [lambda: model.decode(q, z, pool.cache, L), lambda: model.decode(q2, None, pool.cache, L),
             lambda: model.decode(q2[:1].contiguous(), None, pool.cache, few)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    got = _together(calls)
    model.sync_status()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
