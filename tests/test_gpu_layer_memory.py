"""What a model of many layers holds besides its weights: workspaces once, not once a layer."""
import gc

import pytest
import torch

from test_gpu_block_cache import _attend
from test_gpu_w4 import _make

pytestmark = pytest.mark.gpu
MB = 1 << 20


@pytest.fixture(autouse=True)
def no_other_layers(monkeypatch):
    from gated_mla_b200 import api
    monkeypatch.setattr(api, "_layers_scratch", lambda: None)


def _held():
    torch.cuda.synchronize()
    return torch.cuda.memory_allocated()


def test_the_expanded_weight_is_held_once():
    N, H, T = 2048, 32, 300                 # W in fp16: 16 MB; activations 2.4 MB
    layers = [_make(N, H, 64, seed=i) for i in range(5)]
    o = torch.randn(T, H * 128, device="cuda").bfloat16()
    want, base = [], _held()
    for model, w4, _ in layers:
        want.append(model.gate_out_w4(o, w4))
        if len(want) == 1:
            first = _held()
    out = T * N * 2
    assert first - base >= 16 * MB
    assert _held() - first <= 4 * (out + 512) + MB       # the four further outputs, and no workspace
    # layers of other sizes in between: the results are those of the layer alone
    small, sw, g = _make(130, 3, 32, seed=9)
    so = torch.randn(290, 384, device="cuda").bfloat16()
    sy = small.gate_out_w4(so, sw)
    for (model, w4, _), y in zip(layers, want):
        assert torch.equal(model.gate_out_w4(o, w4), y) and torch.equal(small.gate_out_w4(so, sw), sy)
        model.sync_status()


def test_decode_workspaces_are_shared_and_go_with_the_last_layer():
    gc.collect()
    base = _held()
    a = _attend(32, [700, 50], 64, 64, seed=1)
    b = _attend(32, [30, 800], 64, 64, seed=2)
    for model, pool, q, z, L, o in (a, b, a, b):
        assert torch.equal(model.decode(q, z, pool.cache, L), o)
    layers = [a[0], b[0]]
    del a, b, model, pool, q, z, L, o
    gc.collect()
    layers[0].weights.clear(), layers[1].weights.clear()
    with_layers = _held()
    del layers
    gc.collect()
    assert _held() <= base + MB
    assert with_layers - base >= 2 * MB     # at least one decode workspace was still held
