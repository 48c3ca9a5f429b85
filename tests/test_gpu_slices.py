"""Slices that begin off a 16-byte boundary."""
import numpy as np
import pytest
import torch

import operators_ref as R
from test_gpu_block_cache import D, _latents, _model

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("width", [3, 5, 6])
@pytest.mark.parametrize("first", [1, 2, 3])
def test_the_last_sequences_of_a_table_of_odd_width(width, first):
    """Plan, append, project and decode over table[first:]; the rows above it are another batch's."""
    import gated_mla_b200 as gmla
    page, block, B = 16, 16, 4
    g = torch.Generator(device="cuda").manual_seed(width)
    n = lambda *s: (torch.randn(*s, generator=g, device="cuda") / s[-1] ** 0.5).bfloat16()  # noqa: E731
    whole = torch.full((first + B, width), -9, **I32)
    table = whole[first:]
    new, free = torch.tensor([30, 0, 17, 1], **I32), torch.arange(B * width, **I32).flip(0).contiguous()
    plan = gmla.plan_batch(torch.zeros(B, **I32), new, table, free, page, 50)
    want = R.plan([0] * B, new.tolist(), np.full((B, width), -9), free.cpu().numpy(), page, 50)
    assert np.array_equal(table.cpu().numpy(), want["table"]) and np.array_equal(plan.slots.cpu().numpy(), want["slots"])
    assert whole[:first].eq(-9).all()
    gmla.sync_status()
    W = n(16, 128, D), n(16, 128, D)
    q, x = n(B, 16, 128), _latents(48, 2)
    outs = []
    for t in (table, table.clone()):
        model = _model(W_k=W[0], W_v=W[1])
        c = gmla.LatentCache(torch.zeros(B * width, page, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn), t,
                             scales=torch.ones(B * width, 1, device="cuda"), scale_block=block)
        model.cache_append(x, plan.cu_seqlens, plan.seq_lens, c)
        bf16 = gmla.GatedMLA(d_model=256, n_heads=16, d_h=128, d_c=D,
                             weights=dict(W_k=W[0], W_v=W[1], W_q=n(2048, 256), W_c=torch.ones(D, 256).bfloat16().cuda(),
                                          W_g=n(2048, 256)))
        c16 = gmla.LatentCache(torch.zeros(B * width, page, D, dtype=torch.bfloat16, device="cuda"), t)
        bf16.latent_project(torch.ones(50, 256, dtype=torch.bfloat16, device="cuda"), plan.positions, plan.seq_ids, c16)
        outs.append((model.decode(q, None, c, plan.seq_lens), c16.data, bf16.decode(q, None, c16, plan.seq_lens)))
        model.sync_status()
        bf16.sync_status()
    assert outs[0][0].any() and all(torch.equal(a, b) for a, b in zip(*outs))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,first,group", [(129, 1, 0), (129, 3, 32), (512, 2, 128), (777, 5, 0), (1000, 1, 64), (7, 1, 0)])
def test_norm_of_rows_off_a_boundary(dt, d, first, group):
    """x[first:] of odd rows, columns from the first on, a weight that is a slice: as on copies of them."""
    import gated_mla_b200 as gmla
    from test_gpu_add_rms_norm import _check, _inputs
    wide, weight, rw = _inputs(40, d + first, dt)
    w = weight[first:]
    for x, r in ((wide[first:, :d].contiguous().flatten(), rw[first:, :d].contiguous().flatten()),):
        flat, rflat = torch.cat([x.new_zeros(first), x]), torch.cat([r.new_zeros(first), r])
        x1, r1 = flat[first:].view(-1, d), rflat[first:].view(-1, d)
        got = gmla.add_rms_norm(x1, w, r1, fp8_group=group)
        _check(got, x1, w, r1, group)
    x2, r2 = wide[:, first:], rw[:, first:]
    x0, r0, edge = x2.clone(), r2.clone(), wide[:, :first].clone()
    got = gmla.add_rms_norm(x2, w, r2, fp8_group=group, out=x2, residual_out=r2)
    _check(got, x0, w, r0, group)
    assert torch.equal(wide[:, :first], edge)


def test_norm_of_one_row_of_an_odd_matrix():
    import gated_mla_b200 as gmla
    from test_gpu_add_rms_norm import _check, _inputs
    x, w, r = _inputs(9, 515, torch.bfloat16)
    _check(gmla.add_rms_norm(x[7:8], w, r[3:4]), x[7:8], w, r[3:4], 0)
    _check(gmla.add_rms_norm(x[1:], w, r[:-1]), x[1:], w, r[:-1], 0)
