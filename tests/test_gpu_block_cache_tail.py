"""Decode over the block-scaled cache where one token outweighs a long tail whose weights lie below the
grid of the 8-bit products: what the tail adds up to must still be there.

Every row of the tail is the same, at right angles to the query and to the token that dominates, so
the outputs along it are the tail's share alone. The absorbed query, the rows and their scales lie on
the E4M3 grid, and what is left to count is:
  * the last term of a weight w (grid G = 2^-22 of the largest) is rounded with an offset by position;
    over any stretch the offsets below a threshold number within 2 * 4 of an even spread's (the star
    discrepancy of i * 2654435769 / 2^32, i < 2^20, is 4.1 / n; a stretch is a difference of two). A
    CTA's stretch starts anew with a reference of its own, at most three a sequence here: 24 G;
  * fp32 sums: L / 128 tiles of 4 products each in the accumulator and L / 128 terms a thread in the
    softmax sum, each step 2^-23: 2^-23 * 5 L / 128 relative;
  * the weight itself: hardware exponential and logarithm, 2^-18 relative (scores up to 17: of 2^-23
    each, 17 * 1.44 * 2^-23 more);
  * the output in bf16: 2^-8 relative, the merged latent as two bf16 terms: 2^-16."""
import math

import numpy as np
import pytest
import torch

from test_gpu_block_cache import D, _model

pytestmark = pytest.mark.gpu


# 600 sequences over the same rows give each CTA one or two whole sequences. q0 * 16 / sqrt(128) is the dominant token's
# score: 16.0 leaves the tail's weights at 2^-23.08, 17.7 at 2^-25.5, and 14.8 between the grid's points
@pytest.mark.parametrize("H", [16, 32])
@pytest.mark.parametrize("q0", [11.3125, 12.5, 10.4375])
def test_the_tail_under_one_dominant_token_is_not_lost(H, q0):
    import gated_mla_b200 as gmla
    L, page, B = 131072, 128, 600
    rows = torch.zeros(L, D, device="cuda")
    rows[0, :256] = 1
    rows[1:, 256:] = 1
    codes = (rows * 256).to(torch.float8_e4m3fn).view(L // page, page, D)
    cache = gmla.LatentCache(codes, torch.arange(L // page, dtype=torch.int32, device="cuda").repeat(B, 1),
                             scales=torch.full((L // page, 1), 2.0 ** -8, device="cuda"))
    W_k, W_v = torch.zeros(2, H, 128, D, device="cuda")
    W_k[:, 0, :256] = 2.0 ** -4
    half = torch.arange(64, device="cuda")
    W_v[:, half, half] = 1                     # channels 0 .. 63: the dominant token's dims
    W_v[:, 64 + half, 256 + half] = 1          # channels 64 .. 127: the tail's
    model = _model(H, W_k=W_k.bfloat16(), W_v=W_v.bfloat16())
    q = torch.zeros(B, H, 128, device="cuda")
    q[..., 0] = q0
    o = model.decode(q.bfloat16(), None, cache, torch.full((B,), L, dtype=torch.int32, device="cuda"))
    model.sync_status()
    w = math.exp(-q0 * 16 / math.sqrt(128))
    tail = (L - 1) * w
    got = o.double().view(B, H, 2, 64).cpu().numpy()
    rel = 2.0 ** -8 + 2.0 ** -16 + 2.0 ** -18 + 17 * 1.45 * 2.0 ** -23 + 2.0 ** -23 * 5 * L / 128
    head, rest = 1 / (1 + tail), tail / (1 + tail)
    assert np.all(np.abs(got[:, :, 0] - head) <= head * rel)
    assert np.all(np.abs(got[:, :, 1] - rest) <= rest * rel + 24 * 2.0 ** -22), (float(got[:, :, 1].min()), rest)


def test_a_row_of_weight_zero_stays_at_zero():
    """Rows whose weight underflows give nothing, whatever their rounding offset: the result is the dominant row's."""
    import gated_mla_b200 as gmla
    L, page = 5000, 64
    rows = torch.full((L // page + 1, page, D), 1.0, device="cuda")
    rows[0, 0, :256], rows[0, 0, 256:] = 1, 0
    rows.view(-1, D)[1:, :256] = -1
    cache = gmla.LatentCache((rows * 256).to(torch.float8_e4m3fn), torch.arange(len(rows), dtype=torch.int32, device="cuda")[None],
                             scales=torch.full((len(rows), 1), 2.0 ** -8, device="cuda"))
    W_k, W_v = torch.zeros(2, 16, 128, D, device="cuda")
    W_k[:, 0, :256] = 1
    W_v[:, torch.arange(128), 128 + 2 * torch.arange(128)] = 1
    model = _model(W_k=W_k.bfloat16(), W_v=W_v.bfloat16())
    q = torch.zeros(1, 16, 128, device="cuda")
    q[..., 0] = 64
    o = model.decode(q.bfloat16(), None, cache, torch.tensor([L], dtype=torch.int32, device="cuda"))
    assert torch.equal(o.view(16, 2, 64)[:, 0].float(), torch.ones(16, 64, device="cuda")) and not o.view(16, 2, 64)[:, 1].any()
