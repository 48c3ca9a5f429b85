"""A block-scaled layer's decode takes the cache that its cache_append takes: one-byte codes in rows of d_c, on the
queries' device (no GPU needed: the refusals come before any device work)."""
import pytest
import torch

H, D = 16, 512


@pytest.mark.parametrize("data", [torch.zeros(2, 64, D, dtype=torch.bfloat16), torch.zeros(2, 64, 256, dtype=torch.uint8),
                                  torch.zeros(2, 64, D + 64, dtype=torch.uint8)])
@pytest.mark.parametrize("paged", [False, True])
def test_codes_of_another_type_or_width_are_refused(data, paged, monkeypatch):
    import gated_mla_b200 as gmla
    from gated_mla_b200 import api
    from gated_mla_b200 import context_parallel as cp
    calls = []
    monkeypatch.setattr(api, "_stream_of", lambda t: 0)
    for mod in (api, cp):
        monkeypatch.setattr(mod, "_p", lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(api._Scratch, "get", lambda self, key, n, device, stream: torch.zeros(n, dtype=torch.uint8))
    monkeypatch.setattr(api.GatedMLA, "_status_cfg", lambda self, device, staging=False: self.cfg)
    monkeypatch.setattr(api.GatedMLA, "workspace", lambda self, key, n, device: torch.zeros(n, dtype=torch.uint8))
    for name in ("gmla_decode", "gmla_decode_partial"):
        monkeypatch.setattr(api.L, name, lambda *a: calls.append(a) or 0)
    layer = gmla.GatedMLA(d_model=256, n_heads=H, d_h=128, d_c=D, cache_fp8="block", weights={})
    table = torch.zeros(2, 1, dtype=torch.int32) if paged else None
    cache = gmla.LatentCache(data, table, scales=torch.ones(2, 1), scale_block=64)
    q, lens = torch.zeros(2, H, 128, dtype=torch.bfloat16), torch.ones(2, dtype=torch.int32)
    for call in (lambda: layer.decode(q, None, cache, lens), lambda: layer.decode(q, None, cache, lens, ws=torch.zeros(8)),
                 lambda: cp.decode_partial(layer, q, None, cache, lens, lens)):
        with pytest.raises(ValueError, match="codes in rows of"):
            call()
    assert not calls


def test_a_decode_follows_the_layer_s_configuration(monkeypatch):
    """A change of ``layer.cfg`` after the first call reaches the next one."""
    import gated_mla_b200 as gmla
    from gated_mla_b200 import api
    seen = []
    monkeypatch.setattr(api, "_stream_of", lambda t: 0)
    monkeypatch.setattr(api, "_p", lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(api._Scratch, "get", lambda self, key, n, device, stream: torch.zeros(n, dtype=torch.uint8))
    word = torch.zeros(256, dtype=torch.uint8)
    monkeypatch.setattr(api._Scratch, "word", lambda self, key, device: word, raising=False)
    for name in ("gmla_decode", "gmla_gate_out_w4"):
        monkeypatch.setattr(api.L, name, lambda cfg, *a: seen.append((cfg.softmax_scale, cfg.gate_mode, cfg.status)) or 0)
    layer = gmla.GatedMLA(d_model=256, n_heads=H, d_h=128, d_c=D, cache_fp8="block", weights={}, softmax_scale=0.25)
    cache = gmla.LatentCache(torch.zeros(2, 64, D, dtype=torch.uint8), scales=torch.ones(2, 1), scale_block=64)
    w4 = gmla.W4Weight(torch.zeros(256, H * 64, dtype=torch.uint8), torch.zeros(256, H * 2, dtype=torch.bfloat16), 64)
    for scale, mode in ((0.25, 0), (0.5, 1), (2.0, 3)):
        layer.cfg.softmax_scale, layer.cfg.gate_mode = scale, mode
        layer.decode(torch.zeros(2, H, 128, dtype=torch.bfloat16), None, cache, torch.ones(2, dtype=torch.int32))
        layer.gate_out_w4(torch.zeros(1, H * 128, dtype=torch.bfloat16), w4)
        assert seen[-2:] == [(scale, mode, word.data_ptr())] * 2
