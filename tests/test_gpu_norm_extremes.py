"""add_rms_norm where fp32's range ends, as include/gmla.h describes it: an infinity, squares whose sum overflows, and
squares that all underflow under eps = 0. The rows beside them are as they are alone."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [100, 1024])
def test_rows_at_the_ends_of_the_range(dt, d):
    import gated_mla_b200 as gmla
    g = torch.Generator(device="cuda").manual_seed(d)
    x = torch.randn(5, d, generator=g, device="cuda").to(dt)
    alone = gmla.add_rms_norm(x, eps=0.0).out
    x[0, 3] = float("inf")
    x[1] = 1e25 * x[1].sign()
    x[2] = 1e-25 * x[2].sign()
    y = gmla.add_rms_norm(x, eps=0.0).out
    assert y[0, 3].isnan() and not torch.cat([y[0, :3], y[0, 4:]]).any()
    assert not y[1].any()
    assert torch.equal(y[2], float("inf") * x[2].sign())
    assert torch.equal(y[3:], alone[3:])
    z = gmla.add_rms_norm(x, eps=1e-6).out
    assert bool((z[2].float() - 1e-22 * x[2].float().sign()).abs().max() <= 1e-22 * 2.0 ** -7)     # x / sqrt(eps)
