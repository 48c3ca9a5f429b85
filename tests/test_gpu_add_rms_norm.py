"""add_rms_norm against the formula in 64 bits.

Tolerances, relative to |y|: the fp32 part is a sum of d squares taken as at most 32
terms a thread, 5 + 5 levels across lanes and up to 32 warps, a reciprocal root and two
products, each step 2^-24: under 128 * 2^-24. A bf16 result adds half a step, 2^-8. s = x + r
is one fp32 rounding (2^-24 of s) and one when stored. A code stands for y within half an
E4M3 step: 2^-4 of |y|, or 2^-10 of the scale below the normal range."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
F32 = 128 * 2.0 ** -24
STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 0.0}


def _ref(x, w, r, eps):
    s = x.double().cpu() + (r.double().cpu() if r is not None else 0)
    y = s / torch.sqrt((s * s).mean(1, keepdim=True) + eps)
    return s, y * (w.double().cpu() if w is not None else 1)


def _inputs(T, d, dt, residual=True, weight=True, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + T + d)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return n(T, d).to(dt), (1 + 0.3 * n(d)).to(dt) if weight else None, (3 * n(T, d)).to(dt) if residual else None


def _check(got, x, w, r, group, eps=1e-6):
    dt = x.dtype
    s, y = _ref(x, w, r, eps)
    tol = y.abs() * (F32 + STEP[dt]) + 1e-30
    if got.out is not None:
        assert bool(((got.out.double().cpu() - y).abs() <= tol).all())
    if r is not None:
        assert bool(((got.residual.double().cpu() - s).abs() <= s.abs() * (2.0 ** -23 + STEP[dt])).all())
    if not group:
        assert got.codes is None and got.scales is None
        return
    T, d = x.shape
    n = -(-d // group)
    pad = torch.nn.functional.pad(y, (0, n * group - d)).view(T, n, group)
    scale = pad.abs().amax(-1) / 448
    scale = torch.where(scale > 0, scale, torch.ones_like(scale))
    sc = got.scales.double().cpu()
    assert got.scales.shape == (T, n) and bool(((sc - scale).abs() <= scale * (F32 + 2.0 ** -23)).all())
    mine = sc.repeat_interleave(group, 1)[:, :d]
    back = got.codes.float().cpu().double() * mine
    assert bool(((back - y).abs() <= y.abs() * (2.0 ** -4 + F32) + mine * 2.0 ** -10 * (1 + F32)).all())


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d", [(1, 1), (1, 7168), (3, 8), (5, 129), (2, 255), (7, 512), (300, 512), (9, 1000),
                                 (33, 2048), (4, 4099), (500, 4096), (2, 8200), (3, 16384), (2, 20001), (1, 32768)])
def test_norm_with_residual(dt, T, d):
    import gated_mla_b200 as gmla
    x, w, r = _inputs(T, d, dt)
    _check(gmla.add_rms_norm(x, w, r), x, w, r, 0)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("group", [32, 64, 128, 256])
@pytest.mark.parametrize("T,d", [(1, 40), (6, 512), (3, 777), (400, 1024), (2, 7168), (350, 7168), (2, 12344)])
def test_norm_with_codes(dt, group, T, d):
    import gated_mla_b200 as gmla
    x, w, r = _inputs(T, d, dt, residual=d % 2 == 0, weight=T != 3)
    _check(gmla.add_rms_norm(x, w, r, fp8_group=group), x, w, r, group)
    only = gmla.add_rms_norm(x, w, r, fp8_group=group, want_out=False)
    assert only.out is None
    _check(only, x, w, r, group)


def test_rows_of_zeros_and_of_very_different_sizes():
    import gated_mla_b200 as gmla
    x, w, r = _inputs(8, 1024, torch.float32)
    r[0] = -x[0]                       # s = 0: y = 0, scale 1, codes 0
    x[1, 256:512], r[1, 256:512] = 0, 0
    x[2], r[2] = x[2] * 1e-12, r[2] * 1e-12        # below eps
    x[3], r[3] = x[3] * 1e12, r[3] * 1e12
    got = gmla.add_rms_norm(x, w, r, fp8_group=128)
    _check(got, x, w, r, 128)
    assert not got.out[0].any() and not got.codes[0].float().any() and (got.scales[0] == 1).all()
    assert (got.scales[1, 2:4] == 1).all()


def test_strided_rows_and_in_place_results():
    import gated_mla_b200 as gmla
    for dt in (torch.bfloat16, torch.float32):
        for d, width in ((512, 1024), (512, 515), (100, 113)):
            wide, w, rw = _inputs(21, width, dt)
            x, r, w = wide[:, :d], rw[:, :d], w[:d].contiguous()
            x0, r0, rest = x.clone(), r.clone(), wide[:, d:].clone()
            rest_r = rw[:, d:].clone()
            got = gmla.add_rms_norm(x, w, r, out=x, residual_out=r)
            _check(got, x0, w, r0, 0)
            assert torch.equal(wide[:, d:], rest) and torch.equal(rw[:, d:], rest_r)
            assert got.out.data_ptr() == x.data_ptr()


def test_many_rows_match_few_rows_bit_for_bit_within_a_launch_shape():
    """A row's result does not depend on the rows beside it."""
    import gated_mla_b200 as gmla
    x, w, r = _inputs(2000, 1536, torch.bfloat16)
    a = gmla.add_rms_norm(x, w, r)
    b = gmla.add_rms_norm(x[700:1900].contiguous(), w, r[700:1900].contiguous())
    assert torch.equal(a.out[700:1900], b.out) and torch.equal(a.residual[700:1900], b.residual)


def test_a_nan_stays_in_its_row():
    import gated_mla_b200 as gmla
    x, w, r = _inputs(6, 640, torch.bfloat16)
    x[3, 17] = float("nan")
    x[4, 5] = float("inf")
    got = gmla.add_rms_norm(x, w, r)
    ok = [0, 1, 2, 5]
    assert got.out[3].isnan().all() and got.out[4].isnan().any()
    s, y = _ref(x[ok], w, r[ok], 1e-6)
    assert bool(((got.out[ok].double().cpu() - y).abs() <= y.abs() * (F32 + 2.0 ** -8)).all())


def test_refusals():
    import gated_mla_b200 as gmla
    x, w, r = _inputs(4, 64, torch.bfloat16)
    for bad in (lambda: gmla.add_rms_norm(x.half(), w), lambda: gmla.add_rms_norm(x, w.float()),
                lambda: gmla.add_rms_norm(x, w[:32].contiguous()), lambda: gmla.add_rms_norm(x, w, r[:2]),
                lambda: gmla.add_rms_norm(x.t(), None), lambda: gmla.add_rms_norm(x, w, r.float()),
                lambda: gmla.add_rms_norm(x, w, residual_out=r), lambda: gmla.add_rms_norm(x.cpu(), w)):
        with pytest.raises(ValueError):
            bad()
    for kw in (dict(fp8_group=16), dict(eps=float("nan")), dict(eps=-1.0), dict(want_out=False)):
        with pytest.raises(gmla._lib.GmlaError):
            gmla.add_rms_norm(x, w, **kw)
    with pytest.raises(gmla._lib.GmlaError):
        gmla.add_rms_norm(torch.zeros(1, 32776, device="cuda"), None)
    assert gmla.add_rms_norm(x[:0], w).out.shape == (0, 64)


def test_captured_norm():
    import gated_mla_b200 as gmla
    x, w, r = _inputs(16, 2048, torch.bfloat16)
    out, res = torch.empty_like(x), torch.empty_like(x)
    gmla.add_rms_norm(x, w, r, out=out, residual_out=res)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gmla.add_rms_norm(x, w, r, out=out, residual_out=res)
    x2, _, r2 = _inputs(16, 2048, torch.bfloat16, seed=5)
    x.copy_(x2), r.copy_(r2)
    graph.replay()
    torch.cuda.synchronize()
    _check(gmla.NormOut(out, res, None, None), x2, w, r2, 0)
