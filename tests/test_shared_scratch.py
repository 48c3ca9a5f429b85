"""Threads that call one layer on one stream (no GPU needed: the library's calls are replaced by ones that
take their time). A call of several kernels keeps its workspace to itself from the moment it gets it
until its kernels are enqueued."""
import threading
import time

import pytest
import torch

H, DH, D, N = 16, 128, 512, 256


@pytest.fixture
def calls(monkeypatch):
    """The layer's calls on CPU tensors, and how often one got or used a workspace while another was using it."""
    from gated_mla_b200 import api
    state = dict(user=None, clashes=0, done=0)
    held = {}

    def get(self, key, nbytes, device, stream):
        if state["user"] is not None:
            state["clashes"] += 1
        state["user"] = threading.get_ident()
        return held.setdefault(key, torch.zeros(max(nbytes, 256), dtype=torch.uint8))

    def library_call(*a):
        for _ in range(3):           # three kernels
            time.sleep(0.01)
            if state["user"] != threading.get_ident():
                state["clashes"] += 1
                state["user"] = threading.get_ident()
        state["done"] += 1
        state["user"] = None
        return 0
    monkeypatch.setattr(api._Scratch, "get", get)
    monkeypatch.setattr(api, "_stream_of", lambda t: 0)
    monkeypatch.setattr(api, "_p", lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(api.GatedMLA, "cache_append", lambda self, *a: None)
    if hasattr(api.GatedMLA, "_status_cfg"):
        monkeypatch.setattr(api.GatedMLA, "_status_cfg", lambda self, device, staging=False: self.cfg)
    for name in ("gmla_gate_out_w4", "gmla_decode", "gmla_latent_project"):
        monkeypatch.setattr(api.L, name, library_call)
    return state


def _layer():
    import gated_mla_b200 as gmla
    return gmla.GatedMLA(d_model=N, n_heads=H, d_h=DH, d_c=D, cache_fp8="block", weights={})


def _work(layer, what):
    import gated_mla_b200 as gmla
    cache = gmla.LatentCache(torch.zeros(1, 64, D, dtype=torch.uint8), scales=torch.ones(1, 1), scale_block=64)
    lens = torch.ones(1, dtype=torch.int32)
    if what == "gate_out_w4":
        w4 = gmla.W4Weight(torch.zeros(N, H * DH // 2, dtype=torch.uint8), torch.zeros(N, H * DH // 64, dtype=torch.bfloat16), 64)
        return lambda: layer.gate_out_w4(torch.zeros(1, H * DH, dtype=torch.bfloat16), w4)
    if what == "decode":
        return lambda: layer.decode(torch.zeros(1, H, DH, dtype=torch.bfloat16), None, cache, lens)
    return lambda: layer.latent_project(torch.zeros(1, N, dtype=torch.bfloat16), lens, lens, cache,
                                        cu_seqlens=torch.zeros(2, dtype=torch.int32), seq_lens=lens)


def _run(works):
    threads = [threading.Thread(target=lambda w=w: [w() for _ in range(5)]) for w in works]
    for t in threads:
        t.start()
    for t in threads:
        t.join()


@pytest.mark.parametrize("what", ["gate_out_w4", "decode", "latent_project"])
def test_two_threads_of_a_layer_take_turns(calls, what):
    layer = _layer()
    _run([_work(layer, what)] * 2)
    assert calls["done"] == 10 and calls["clashes"] == 0


@pytest.mark.parametrize("what", ["gate_out_w4", "decode", "latent_project"])
def test_two_layers_in_two_threads_take_turns(calls, what):
    """Layers share workspaces."""
    _run([_work(_layer(), what), _work(_layer(), what)])
    assert calls["done"] == 10 and calls["clashes"] == 0


def test_layers_share_their_workspaces_while_there_are_layers(monkeypatch):
    import gc

    from gated_mla_b200 import api
    monkeypatch.setattr(api, "_layers_scratch", lambda: None)
    a, b = _layer(), _layer()
    assert a._scratch is b._scratch and a._status is not b._status
    ref = api._layers_scratch
    del a
    gc.collect()
    assert ref() is b._scratch
    del b
    gc.collect()
    assert ref() is None
