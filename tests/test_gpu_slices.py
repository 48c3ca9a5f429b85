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
