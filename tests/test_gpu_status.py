"""Faults that kernels report: those of captured calls can be read, they stay until they are cleared, they go
once they are, and each layer has its own."""
import pytest
import torch

from test_gpu_block_cache import D, Pool, _attend, _latents, _model

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")


def _raises(sync):
    import gated_mla_b200 as gmla
    for _ in range(2):
        with pytest.raises(gmla._lib.GmlaError) as e:
            sync()
        assert e.value.status == gmla._lib.GMLA_ERR_DEVICE_RANGE


@pytest.mark.parametrize("first_call_is_captured", [False, True])
def test_a_captured_plan_that_does_not_fit(first_call_is_captured, monkeypatch):
    import gated_mla_b200 as gmla
    from gated_mla_b200 import api
    monkeypatch.setattr(api, "_scratch", api._Scratch())
    cached, new = torch.tensor([15, 16], **I32), torch.tensor([2, 1], **I32)
    table, free = torch.tensor([[7, -1], [8, -1]], **I32), torch.tensor([3], **I32)     # two pages are needed
    if not first_call_is_captured:
        gmla.plan_batch(cached, torch.zeros_like(new), table, free, 16, 4)
        gmla.sync_status()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan = gmla.plan_batch(cached, new, table, free, 16, 4)
    gmla.sync_status()
    graph.replay()
    _raises(gmla.sync_status)
    assert plan.seq_lens.tolist() == [0, 0]
    new.copy_(torch.tensor([1, 1], **I32))             # one page
    graph.replay()                                     # a good replay does not hide the one before
    _raises(gmla.sync_status)
    gmla.clear_status()
    graph.replay()
    gmla.sync_status()
    assert plan.seq_lens.tolist() == [16, 17] and table.tolist() == [[7, -1], [8, 3]]


def test_an_eager_plan_that_does_not_fit_is_forgotten_when_cleared():
    import gated_mla_b200 as gmla
    gmla.clear_status()
    one = torch.tensor([1], **I32)
    gmla.plan_batch(one, one, torch.full((1, 1), 5, **I32), one[:0], 1, 4)
    _raises(gmla.sync_status)
    gmla.clear_status()
    gmla.sync_status()


@pytest.mark.parametrize("what", ["append", "decode"])
@pytest.mark.parametrize("first_call_is_captured", [False, True])
def test_a_fault_in_a_captured_call_of_a_layer(what, first_call_is_captured):
    import gated_mla_b200 as gmla
    made, pool, q, z, L, o = _attend(16, [40, 20], 64, 32, seed=3)
    layer = gmla.GatedMLA(d_model=256, n_heads=16, d_h=128, d_c=D, cache_fp8="block", weights=made.weights)
    cu, lens, x = torch.tensor([0, 1, 2], **I32), torch.tensor([41, 21], **I32), _latents(2, 5)

    def call():
        return layer.cache_append(x, cu, lens, pool.cache) if what == "append" else layer.decode(q, z, pool.cache, L)
    if not first_call_is_captured:
        call()
        layer.sync_status()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    graph.replay()
    layer.sync_status()
    scale = pool.cache.scales[int(pool.table[0, 0]), 1].clone()
    pool.cache.scales[int(pool.table[0, 0]), 1] = float("nan")
    graph.replay()
    pool.cache.scales[int(pool.table[0, 0]), 1] = scale
    graph.replay()
    _raises(layer.sync_status)
    made.sync_status()                                 # another layer over the same cache, its own status
    layer.clear_status()
    graph.replay()
    layer.sync_status()


def test_clearing_covers_the_calls_over_a_bf16_cache():
    import gated_mla_b200 as gmla
    W = torch.zeros(16, 128, D, dtype=torch.bfloat16, device="cuda")
    layer = gmla.GatedMLA(d_model=256, n_heads=16, d_h=128, d_c=D, weights=dict(W_k=W, W_v=W))
    cache = gmla.LatentCache(torch.zeros(1, 8, D, dtype=torch.bfloat16, device="cuda"))
    layer.decode(torch.zeros(1, 16, 128, dtype=torch.bfloat16, device="cuda"), None, cache, torch.tensor([9], **I32))
    _raises(layer.sync_status)
    layer.clear_status()
    layer.sync_status()


def test_a_prompt_s_projection_reports_into_the_layer(monkeypatch):
    """latent_project over a block-scaled cache: the append behind it, more rows than the cache has."""
    import gated_mla_b200 as gmla
    g = torch.Generator(device="cuda").manual_seed(0)
    n = lambda *s: (torch.randn(*s, generator=g, device="cuda") / s[-1] ** 0.5).bfloat16()  # noqa: E731
    w = dict(W_q=n(2048, 256), W_c=n(D, 256), W_g=n(2048, 256), W_k=n(16, 128, D), W_v=n(16, 128, D))
    layer = gmla.GatedMLA(d_model=256, n_heads=16, d_h=128, d_c=D, cache_fp8="block", weights=w)
    pool = Pool(1, 32, 16, 16)
    none = torch.zeros(40, **I32)
    layer.latent_project(n(40, 256), none, none, pool.cache, cu_seqlens=torch.tensor([0, 40], **I32),
                         seq_lens=torch.tensor([40], **I32))
    _raises(layer.sync_status)


def test_status_words_made_under_capture_are_zero_and_apart():
    from gated_mla_b200 import _lib as lib
    graph, t = torch.cuda.CUDAGraph(), torch.zeros(4, device="cuda")
    with torch.cuda.graph(graph):
        t += 1
        words = [lib.gmla_status_word() for _ in range(600)]       # several slabs
    graph.replay()
    torch.cuda.synchronize()
    assert t.tolist() == [1] * 4
    assert len(set(words)) == 600 and all(a % 256 == 0 for a in words)
    for a in words[:3] + words[255:258] + words[-1:]:
        lib.check(lib.gmla_sync_status(a, None), "word")
