"""gate_out_w4 on infinite and very large activations, against the definition in 64 bits: an infinity
gives the infinity of w's sign, w = 0 or two signs give NaN, and a finite result is finite however
large its terms are. The tolerance of a finite element is that of test_gpu_w4.py."""
import numpy as np
import pytest
import torch

import operators_ref as R
from test_gpu_w4 import _make

pytestmark = pytest.mark.gpu
BIG = 3.0e38
# a single tile of 8, 16 and 32 tokens, several of 32, and (above 256) the product over fp16 rows
TOKENS = [1, 5, 13, 29, 70, 256, 300]


def _want(w4, group, o, gate=None):
    """(y, sum |w a|, sum scale |a|) in 64 bits, infinities by the rules of IEEE arithmetic."""
    W = R.w4_dense(w4.codes.cpu().numpy(), w4.scales.float().cpu().numpy(), group)
    a = o.double().cpu().numpy()
    if gate is not None:
        a = a * gate
    y = np.empty((len(a), len(W)))
    with np.errstate(invalid="ignore"):
        for t in range(len(a)):
            if np.isfinite(a[t]).all():
                y[t] = W @ a[t]
            else:                # a matrix product may skip zeros: term by term
                y[t] = (W * a[t]).sum(1)
    fin = np.where(np.isfinite(a), a, 0)
    s = np.repeat(w4.scales.double().cpu().numpy(), group, axis=1)
    return y, np.abs(fin) @ np.abs(W).T, np.abs(fin) @ s.T


def _check(y, ref, S, Ss, K, many, top, Wsum, gated=False):
    got = y.double().cpu().numpy()
    fin = np.isfinite(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    assert np.array_equal(got[~fin & ~np.isnan(ref)], ref[~fin & ~np.isnan(ref)])
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -23 * ((K / 16 + 64) * S + 12 * 144 * Ss)
    if many:
        tol = tol + 2.0 ** -12 * S + 2.0 ** -39 * top[:, None] * Wsum
    if gated:
        tol = tol + (2.0 ** -8 + 2.0 ** -20) * S
    assert np.all(np.abs(got[fin] - ref[fin]) <= tol[fin])


def _Wsum(w4, group):
    return np.abs(R.w4_dense(w4.codes.cpu().numpy(), w4.scales.float().cpu().numpy(), group)).sum(1)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T", TOKENS)
def test_infinite_activations(T, group):
    N, H = 130, 5
    K = H * 128
    model, w4, g = _make(N, H, group)
    o = torch.randn(T, K, generator=g, device="cuda").to(torch.bfloat16)
    o[0, 3] = float("inf")
    if T > 4:
        o[1, K - 1] = float("-inf")
        o[3, 5], o[3, 400] = float("inf"), float("-inf")
        o[4, 7] = float("nan")
    y = model.gate_out_w4(o, w4)
    model.sync_status()
    ref, S, Ss = _want(w4, group, o)
    assert np.isinf(ref[0]).any() and np.isnan(ref[0]).any()       # some codes are 8, a weight of 0
    top = np.nan_to_num(o.double().cpu().abs().numpy(), nan=0, posinf=0).max(1)
    _check(y, ref, S, Ss, K, T > 256, top, _Wsum(w4, group))


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("T", TOKENS)
def test_activations_near_the_largest_number(T, group):
    """|a| up to 3e38, whose products pass fp32's range before they are scaled; y stays below it."""
    N, H = 97, 5
    K = H * 128
    model, w4, g = _make(N, H, group)
    w4.scales[:] = (w4.scales.float() * 2.0 ** -20).bfloat16()
    o = torch.randn(T, K, generator=g, device="cuda")
    o[0] = torch.where(torch.arange(K, device="cuda") % 2 == 0, BIG, -BIG) * torch.rand(K, generator=g, device="cuda")
    if T > 4:
        o[2, 17] = BIG                     # one large element among ordinary ones
        o[3] *= 2.0 ** 100                 # elements on both sides of the kernel's threshold
        o[4] *= 2.0 ** 103
    o = o.to(torch.bfloat16)
    assert o.isfinite().all()
    y = model.gate_out_w4(o, w4)
    model.sync_status()
    ref, S, Ss = _want(w4, group, o)
    assert np.abs(ref).max() < 1e38
    _check(y, ref, S, Ss, K, T > 256, o.double().cpu().abs().amax(1).numpy(), _Wsum(w4, group))


@pytest.mark.parametrize("gate", ["channel", "head"])
@pytest.mark.parametrize("T", [2, 40])
def test_infinite_activations_behind_a_gate(gate, T):
    N, H, group = 64, 4, 64
    K = H * 128
    model, w4, g = _make(N, H, group, gate=gate)
    o = torch.randn(T, K, generator=g, device="cuda").to(torch.bfloat16)
    z = torch.randn(T, model.G, generator=g, device="cuda")
    o[1, 200] = float("inf")
    y = model.gate_out_w4(o, w4, z)
    model.sync_status()
    ref, S, Ss = _want(w4, group, o, R.gate_values(z.double().cpu().numpy(), gate, H, 128))
    _check(y, ref, S, Ss, K, False, None, None, gated=True)


def test_an_infinity_leaves_the_rows_beside_it_as_they_were():
    model, w4, g = _make(300, 8, 64)
    o = torch.randn(32, 1024, generator=g, device="cuda").to(torch.bfloat16)
    y = model.gate_out_w4(o, w4)
    o2 = o.clone()
    o2[9, 100], o2[20, 5] = float("inf"), BIG
    y2 = model.gate_out_w4(o2, w4)
    keep = [t for t in range(32) if t not in (9, 20)]
    assert torch.equal(y2[keep], y[keep])
    assert not y2[9].isfinite().any()
