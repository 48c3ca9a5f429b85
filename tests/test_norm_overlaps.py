"""add_rms_norm's outputs may be its inputs, rows that lie side by side are apart, and any other overlap is refused:
one thread would read what another has already written."""
import pytest
import torch

P = 1 << 20     # an aligned address that no accepted call gets to use
T, D, S = 4, 64, 128


def _call(**kw):
    from gated_mla_b200 import _lib as L
    M = 1 << 14
    a = dict(dtype=0, x=P, x_stride=S, residual=P + M, residual_stride=S, weight=P + 2 * M, eps=1e-6, T=T, d=D,
             residual_out=P + 3 * M, residual_out_stride=S, out=P + 4 * M, out_stride=S, codes=P + 5 * M, scales=P + 6 * M,
             group=32, stream=None)
    a.update(kw)
    return L.gmla_add_rms_norm(*a.values()), L.lib.gmla_last_error().decode()


M, R = 1 << 14, 2 * S          # between the arrays, and between the rows of one, in bytes


# (none of these reaches a launch)
@pytest.mark.parametrize("kw,names", [
    (dict(out=P + R), ("out", "x")), (dict(out=P - R), ("out", "x")), (dict(out=P + 16), ("out", "x")),
    (dict(out=P, out_stride=2 * S), ("out", "x")), (dict(out=P, out_stride=D), ("out", "x")),
    (dict(out=P + M + 3 * R), ("out", "residual")), (dict(residual_out=P + R), ("residual_out", "x")),
    (dict(residual_out=P + M - 64), ("residual_out", "residual")),
    (dict(residual_out=P + 2 * M), ("residual_out", "weight")), (dict(out=P + 2 * M - R), ("out", "weight")),
    (dict(out=P + 3 * M), ("residual_out", "out")), (dict(out=P + 3 * M + R), ("residual_out", "out")),
    (dict(out=P + 3 * M + 64), ("residual_out", "out")), (dict(codes=P), ("codes", "x")), (dict(codes=P + 4 * M + 64), ("out", "codes")),
    (dict(scales=P + 5 * M + 16), ("codes", "scales")), (dict(scales=P + 2 * M + 64), ("scales", "weight")),
    (dict(T=1, out=P + 16), ("out", "x")), (dict(out=P, residual_out=P), ("residual_out", "out"))])
def test_refused(kw, names):
    from gated_mla_b200 import _lib as L
    status, message = _call(**kw)
    assert status == L.GMLA_ERR_INVALID_ARG and all(n in message for n in names) and "overlap" in message


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,d", [(1, 512), (40, 512), (700, 136)])
def test_taken(dt, rows, d):
    """In place, and side by side in one matrix."""
    import gated_mla_b200 as gmla
    g = torch.Generator(device="cuda").manual_seed(rows)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dt)  # noqa: E731
    x, r, w = n(rows, d), n(rows, d), n(d)
    want = gmla.add_rms_norm(x, w, r)
    for out, res in (("x", "r"), ("r", "x"), ("x", None), ("r", None), (None, "x"), (None, "r")):
        a = dict(x=x.clone(), r=r.clone())
        got = gmla.add_rms_norm(a["x"], w, a["r"], out=a.get(out), residual_out=a.get(res))
        assert torch.equal(got.out, want.out) and torch.equal(got.residual, want.residual), (out, res)
    wide = n(rows + 1, 4 * d + 8)
    a = [wide[:rows, i * d:(i + 1) * d] for i in range(4)]
    a[0].copy_(x), a[1].copy_(r)
    edge = wide[:, 4 * d:].clone()
    got = gmla.add_rms_norm(a[0], w, a[1], out=a[3], residual_out=a[2])
    assert torch.equal(got.out, want.out) and torch.equal(a[2], want.residual) and torch.equal(a[0], x)
    assert torch.equal(wide[:, 4 * d:], edge)
