"""A wait that runs out in the FP8 attention (see test_gpu_timeout.py): the block leaves through its abort path, the
status says so, and the same layer decodes correctly right after it is cleared. 16 heads (one issuing warp, two blocks
an SM) and 32 heads (two issuing warps) over a block-scaled cache, and one scale for the whole cache."""
import time

import pytest
import torch

from test_gpu_block_cache import D, _attend

pytestmark = pytest.mark.gpu


def _stall(model, call, want):
    from gated_mla_b200 import _lib
    _lib.check(_lib.gmla_test_stall_next_decode(1), "arm the stall")
    t0 = time.perf_counter()
    call()
    with pytest.raises(_lib.GmlaError) as e:
        model.sync_status()
    waited = time.perf_counter() - t0
    assert e.value.status == _lib.GMLA_ERR_TIMEOUT
    assert 0.9 <= waited < 10, waited
    model.clear_status()
    assert torch.equal(call(), want)
    model.sync_status()


# sequences of one tile, of many in one block, and spread over blocks
@pytest.mark.parametrize("H", [16, 32])
@pytest.mark.parametrize("lens", [[5], [300, 1, 129, 2000], [40000]])
def test_block_scales(H, lens):
    model, pool, q, z, L, o = _attend(H, lens, 64, 64, seed=H)
    _stall(model, lambda: model.decode(q, z, pool.cache, L), o)


@pytest.mark.parametrize("H", [16, 32])
def test_one_scale(H):
    import gated_mla_b200 as gmla
    g = torch.Generator(device="cuda").manual_seed(H)
    n = lambda *s: (torch.randn(*s, generator=g, device="cuda") / s[-1] ** 0.5).bfloat16()  # noqa: E731
    model = gmla.GatedMLA(d_model=256, n_heads=H, d_h=128, d_c=D, cache_fp8=True, cache_scale=1 / 64,
                          weights=dict(W_k=n(H, 128, D), W_v=n(H, 128, D)))
    cache = gmla.LatentCache((64 * torch.randn(3, 2000, D, generator=g, device="cuda")).clamp(-448, 448).to(torch.float8_e4m3fn))
    q, L = n(3, H, 128), torch.tensor([300, 1, 2000], dtype=torch.int32, device="cuda")
    _stall(model, lambda: model.decode(q, None, cache, L), model.decode(q, None, cache, L))
