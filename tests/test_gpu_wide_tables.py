"""A block table whose width times the page size passes 32 bits: its sequences are as long as their lengths say."""
import pytest
import torch

from test_gpu_block_cache import D, _latents, _model

pytestmark = pytest.mark.gpu


# 2^20 + 1 pages of 4096 rows: 2^32 + 4096 rows, of which 32 bits keep 4096; 2^19 pages: a negative number
@pytest.mark.parametrize("width", [1 << 19, 1 << 20, (1 << 20) + 1])
@pytest.mark.parametrize("cache", ["block", "bf16", "fp32"])
def test_append_and_decode(cache, width):
    import gated_mla_b200 as gmla
    page, L = 4096, 5000
    g = torch.Generator(device="cuda").manual_seed(width)
    dt = torch.float32 if cache == "fp32" else torch.bfloat16
    W = (torch.randn(2, 16, 128, D, generator=g, device="cuda") / D ** 0.5).to(dt)
    q = torch.randn(1, 16, 128, generator=g, device="cuda").to(dt)
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    outs = []
    for M in (width, 2):
        table = torch.full((1, M), -1, dtype=torch.int32, device="cuda")
        table[0, :2] = torch.tensor([2, 0], dtype=torch.int32)
        if cache == "block":
            model = _model(W_k=W[0], W_v=W[1])
            c = gmla.LatentCache(torch.zeros(3, page, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn), table,
                                 scales=torch.ones(3, page // 64, device="cuda"))
            model.cache_append(_latents(L, 5), torch.tensor([0, L], dtype=torch.int32, device="cuda"), lens, c)
        else:
            model = gmla.GatedMLA(d_model=256, n_heads=16, d_h=128, d_c=D, dtype=dt, weights=dict(W_k=W[0], W_v=W[1]))
            c = gmla.LatentCache(_latents(3 * page, 5).to(dt).view(3, page, D), table)
        outs.append(model.decode(q, None, c, lens))
        model.sync_status()
    assert bool(outs[0].any()) and torch.equal(outs[0], outs[1])


@pytest.mark.parametrize("length", [2 ** 31 - 1, 2 ** 31 - 128, 2 ** 31 - 255])
@pytest.mark.parametrize("cache", ["block", "bf16"])
def test_lengths_that_round_up_past_32_bits_are_reported(cache, length):
    import gated_mla_b200 as gmla
    page, M = 4096, 1 << 19
    W = torch.zeros(16, 128, D, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(1, M, dtype=torch.int32, device="cuda")
    lens = torch.tensor([length], dtype=torch.int32, device="cuda")
    if cache == "block":
        model = _model(W_k=W, W_v=W)
        c = gmla.LatentCache(torch.zeros(1, page, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn), table,
                             scales=torch.ones(1, page // 64, device="cuda"))
    else:
        model = gmla.GatedMLA(d_model=256, n_heads=16, d_h=128, d_c=D, weights=dict(W_k=W, W_v=W))
        c = gmla.LatentCache(torch.zeros(1, page, D, dtype=torch.bfloat16, device="cuda"), table)
    calls = [lambda: model.decode(torch.zeros(1, 16, 128, dtype=torch.bfloat16, device="cuda"), None, c, lens)]
    if cache == "block":
        calls.append(lambda: model.cache_append(_latents(1, 1), torch.tensor([0, 1], dtype=torch.int32, device="cuda"), lens, c))
    for call in calls:
        call()
        with pytest.raises(gmla._lib.GmlaError) as e:
            model.sync_status()
        assert e.value.status == gmla._lib.GMLA_ERR_DEVICE_RANGE
        model.clear_status()
    assert not c.data.view(torch.uint8).any()
