"""cache_append refuses what it cannot continue: the fault is reported, nothing of it is written, and the
other sequences get their rows."""
import numpy as np
import pytest
import torch

from test_gpu_block_cache import D, Pool, _latents, _model

pytestmark = pytest.mark.gpu


def _reported(model):
    import gated_mla_b200 as gmla
    with pytest.raises(gmla._lib.GmlaError) as e:
        model.sync_status()
    assert e.value.status == gmla._lib.GMLA_ERR_DEVICE_RANGE


# blocks of 8 are taken by a warp, of 64 by a block of threads
@pytest.mark.parametrize("block", [2, 8, 64])
@pytest.mark.parametrize("scale", [float("nan"), 0.0, -1.0, 2.0 ** 40, 2.0 ** -40, float("inf"), -float("inf")])
@pytest.mark.parametrize("paged", [True, False])
def test_a_block_held_under_a_bad_scale_is_left_and_reported(block, scale, paged):
    """Continuing such a block would give its codes a valid scale, and hide the fault from the next decode."""
    model = _model()
    pool = Pool(3, 256, 64 if paged else 0, block)
    held = block + 1                      # the block at positions block .. 2 block - 1 holds one row
    pool.append(model, _latents(3 * held, 1), [held] * 3, [held] * 3)
    pool.same()
    model.sync_status()
    at = pool.block_of(1, block)
    pool.cache.scales.view(-1)[at] = scale
    pool.scales[at] = scale
    codes, scales = pool.codes.copy(), pool.scales.copy()
    x = _latents(6 * block, 2)
    n = 2 * block                         # the rest of that block, a whole one, and one row of the next
    cu = torch.tensor([0, n, 2 * n, 3 * n], dtype=torch.int32, device="cuda")
    model.cache_append(x, cu, torch.full((3,), held + n, dtype=torch.int32, device="cuda"), pool.cache)
    _reported(model)
    import operators_ref as R
    with np.errstate(all="ignore"):       # the block in question is put back below
        R.append(pool.codes, pool.scales, pool.row_of, pool.block_of, x.double().cpu().numpy(), cu.tolist(), [held + n] * 3,
                 block)
    # the block in question is as it was, the later blocks of the sequence are appended
    first = pool.row_of(1, block)
    pool.codes[first:first + block], pool.scales[at] = codes[first:first + block], scales[at]
    pool.same()


def test_the_decode_after_it_still_sees_the_fault():
    model = _model(W_k=torch.zeros(16, 128, D, dtype=torch.bfloat16, device="cuda"),
                   W_v=torch.zeros(16, 128, D, dtype=torch.bfloat16, device="cuda"))
    pool = Pool(1, 64, 64, 64)
    pool.append(model, _latents(3, 1), [3], [3])
    pool.cache.scales[int(pool.table[0, 0]), 0] = float("nan")
    lens = torch.tensor([4], dtype=torch.int32, device="cuda")
    model.cache_append(_latents(1, 2), torch.tensor([0, 1], dtype=torch.int32, device="cuda"), lens, pool.cache)
    _reported(model)
    other = _model(W_k=model.weights["W_k"], W_v=model.weights["W_v"])
    other.decode(torch.zeros(1, 16, 128, dtype=torch.bfloat16, device="cuda"), None, pool.cache, lens)
    _reported(other)


def test_offsets_past_the_rows_are_reported_when_the_batch_is_a_slice_too():
    """A slice of a packed batch: its offsets start behind 0, and end behind the rows that were given."""
    model = _model()
    pool = Pool(2, 64, 16, 16)
    cu = torch.tensor([2, 4, 9], dtype=torch.int32, device="cuda")
    model.cache_append(_latents(6, 1), cu, torch.tensor([2, 5], dtype=torch.int32, device="cuda"), pool.cache)
    _reported(model)
