"""A padded plan (n_tokens above the sum of the new lengths, as a captured step of fixed size has it)
goes through latent_project over every cache: live rows land in the cache, padding touches nothing
and is no fault, and any other index outside the cache still is one."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
N, H, DH, D, PAGE, M = 256, 16, 128, 512, 64, 4
NEW = [1, 70, 0, 33]


def _layer(kind, rope=0):
    import gated_mla_b200 as gmla
    dt = torch.float32 if kind == "fp32" else torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(3)
    n = lambda *s: (torch.randn(*s, generator=g, device="cuda") / s[-1] ** 0.5).to(dt)  # noqa: E731
    w = dict(W_q=n(H * DH, N), W_c=n(D, N), W_g=n(H * DH, N), W_k=n(H, DH, D), W_v=n(H, DH, D))
    if rope:
        w.update(W_kr=n(rope, N), W_qr=n(H * rope, N))
    kw = dict(cache_fp8=True, cache_scale=1 / 64) if kind == "fp8" else {}
    return gmla.GatedMLA(d_model=N, n_heads=H, d_h=DH, d_c=D, d_rope=rope, dtype=dt, weights=w, **kw), g, dt


def _cache(kind, dt, row, pages):
    if kind == "fp8":
        return torch.full((pages, PAGE, row), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    return torch.full((pages, PAGE, row), float("nan"), dtype=dt, device="cuda")


# 104 live tokens: padded to 120 (few tokens) and 300 (many)
@pytest.mark.parametrize("kind,rope", [("bf16", 0), ("bf16", 64), ("fp8", 0), ("fp32", 0)])
@pytest.mark.parametrize("T", [sum(NEW), 120, 300])
def test_padding_is_neither_cached_nor_a_fault(kind, rope, T):
    import gated_mla_b200 as gmla
    layer, g, dt = _layer(kind, rope)
    B, live, row = len(NEW), sum(NEW), D + rope
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.full((B, M), -1, **i32)
    pages = B * M
    free = torch.randperm(pages, generator=g, device="cuda").int()
    plan = gmla.plan_batch(torch.zeros(B, **i32), torch.tensor(NEW, **i32), table, free, PAGE, T)
    assert plan.positions[live:].eq(-1).all() and plan.seq_ids[live:].eq(-1).all()
    cache = gmla.LatentCache(_cache(kind, dt, row, pages), table)
    x = torch.randn(T, N, generator=g, device="cuda").to(dt)
    q, z = layer.latent_project(x, plan.positions, plan.seq_ids, cache)
    layer.sync_status()
    gmla.sync_status()
    data = cache.data.float().view(-1, row).cpu().numpy()
    slots = plan.slots[:live].cpu().numpy()
    written = np.isfinite(data).all(1)
    want = np.zeros(len(data), bool)
    want[slots] = True
    assert np.array_equal(written, want) and np.isnan(data[~want]).all()
    c = x[:live].double().cpu().numpy() @ layer.weights["W_c"].double().cpu().numpy().T
    got = data[slots][:, :D] * (1 / 64 if kind == "fp8" else 1)
    mag = np.abs(x[:live].double().cpu().numpy()) @ np.abs(layer.weights["W_c"].double().cpu().numpy().T)
    # fp32 sums over N terms; half a step of bf16 or of E4M3 (half a subnormal step, 2^-10 of the scale, below its range)
    tol = 2.0 ** -23 * N * mag + {"bf16": 2.0 ** -8, "fp32": 2.0 ** -23, "fp8": 2.0 ** -4}[kind] * np.abs(c) * (1 + 2.0 ** -8)
    if kind == "fp8":
        tol = tol + 2.0 ** -10 / 64
        c = np.clip(c, -448 / 64, 448 / 64)
    assert np.all(np.abs(got - c) <= tol)
    assert q.shape[0] == T and z.shape[0] == T and bool(q[:live].isfinite().all())


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [4, 300])
@pytest.mark.parametrize("pos,seq", [(-1, 0), (0, -1), (-2, -1), (-1, -2), (M * PAGE, 0), (0, len(NEW))])
def test_other_indices_outside_the_cache_are_reported(kind, T, pos, seq):
    import gated_mla_b200 as gmla
    layer, g, dt = _layer(kind)
    table = torch.arange(len(NEW) * M, dtype=torch.int32, device="cuda").view(len(NEW), M)
    cache = gmla.LatentCache(_cache(kind, dt, D, len(NEW) * M), table)
    positions = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    seqs = positions.clone()
    positions[2], seqs[2] = pos, seq
    layer.latent_project(torch.randn(T, N, generator=g, device="cuda").to(dt), positions, seqs, cache)
    with pytest.raises(gmla._lib.GmlaError) as e:
        layer.sync_status()
    assert e.value.status == gmla._lib.GMLA_ERR_DEVICE_RANGE
    assert bool(cache.data.isnan().all())


def test_captured_padded_step_over_a_bf16_cache():
    """One graph of 8 token rows, replayed on batches of other lengths."""
    import gated_mla_b200 as gmla
    layer, g, dt = _layer("bf16")
    B, T, pages = 4, 8, 16
    i32 = dict(dtype=torch.int32, device="cuda")
    cached, new, table = torch.zeros(B, **i32), torch.tensor([1, 1, 0, 1], **i32), torch.full((B, M), -1, **i32)
    free = torch.arange(pages, **i32)
    cache = gmla.LatentCache(_cache("bf16", dt, D, pages), table)
    x = torch.randn(T, N, generator=g, device="cuda").to(dt)

    def step():
        plan = gmla.plan_batch(cached, new, table, free, PAGE, T)
        q, z = layer.latent_project(x, plan.positions, plan.seq_ids, cache)
        return plan, layer.decode(q[:B].contiguous(), z[:B].contiguous(), cache, plan.seq_lens)
    step()
    torch.cuda.synchronize()
    table.fill_(-1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan, o = step()
    for lens in ([2, 3, 0, 1], [0, 0, 0, 0], [8, 0, 0, 0], [2, 2, 2, 2]):
        table.fill_(-1)
        cache.data.fill_(float("nan"))
        new.copy_(torch.tensor(lens, **i32))
        graph.replay()
        torch.cuda.synchronize()
        layer.sync_status()
        gmla.sync_status()
        written = cache.data.view(-1, D).isfinite().all(1).nonzero()[:, 0]
        assert torch.equal(written, plan.slots[:sum(lens)].sort().values)
        assert bool(o.isfinite().all()) and not o[torch.tensor(lens) == 0].any()
