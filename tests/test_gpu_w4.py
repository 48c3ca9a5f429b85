"""gate_out_w4: y = W [gate ⊙ o] with W in 4 bits, against 64 bits.

Tolerance of an element, with S = sum_k |w_k| |a_k|: up to 256 tokens the codes are exact, the gated
activation is rounded to bf16 (2^-8 S, only where a gate is applied; the sigmoid itself
2^-20 S), the fp32 sums run over at most K terms of which each step drops 2^-23 at most, in
chains of K / 16 (2^-23 (K / 16 + 64) S), and the result is rounded to bf16 (2^-8 |y|). A group's
products are taken with 128 + v and corrected by 136 times the group's sum: up to 8 steps and
the correction, each on at most 144 sum scale |a| (2^-23 * 12 * 144 sum_k scale |a|). Above 256
tokens activations and weights are fp16 numbers under a power of two for each row: weights exact (the
scales of a row lie within 2^28 of one another), activations rounded to 2^-12, or to half a
subnormal step, 2^-25 with the row's largest at 2^14: 2^-39 max|a| sum_k |w_k|."""
import numpy as np
import pytest
import torch

import operators_ref as R

pytestmark = pytest.mark.gpu


def _make(N, H, group, d_h=128, gate="channel", topk=0, seed=0):
    import gated_mla_b200 as gmla
    g = torch.Generator(device="cuda").manual_seed(seed + N + H)
    K = H * d_h
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = (torch.rand(N, K // group, generator=g, device="cuda") + 0.1).to(torch.bfloat16) / K ** 0.5
    scales = scales.to(torch.bfloat16)
    model = gmla.GatedMLA(d_model=N, n_heads=H, d_h=d_h, d_c=512, gate_mode=gate, weights={}, gate_topk=topk)
    return model, gmla.W4Weight(codes, scales, group), g


def _run(N, H, group, T, d_h=128, gate=None, topk=0, seed=0, rows=None):
    model, w4, g = _make(N, H, group, d_h, gate or "channel", topk, seed)
    K = H * d_h
    o = torch.randn(T, K, generator=g, device="cuda").to(torch.bfloat16)
    z = 1.5 * torch.randn(T, model.G, generator=g, device="cuda") if gate else None
    y = model.gate_out_w4(o, w4, z)
    model.sync_status()
    W = torch.from_numpy(R.w4_dense(w4.codes.cpu().numpy(), w4.scales.float().cpu().numpy(), group))
    a = o.double().cpu()
    if gate:
        a = a * torch.from_numpy(R.gate_values(z.double().cpu().numpy(), gate, H, d_h, topk))
    ref, S = a @ W.t(), a.abs() @ W.abs().t()
    tol = 2.0 ** -8 * ref.abs() + 2.0 ** -23 * (K / 16 + 64) * S
    if T > 256:
        tol += 2.0 ** -12 * S + 2.0 ** -39 * a.abs().amax(1, keepdim=True) * W.abs().sum(1)
    elif gate:
        tol += 2.0 ** -8 * S
    if gate:
        tol += 2.0 ** -20 * S
    sc = w4.scales.double().cpu().repeat_interleave(group, 1)
    tol += 2.0 ** -23 * 12 * 144 * (a.abs() @ sc.t())
    err = (y.double().cpu() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    assert float((y.double().cpu() - ref).norm() / ref.norm()) < 5e-3
    return model, w4, o, z, y


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 17, 32, 33, 64, 65, 130, 300])
def test_tokens_and_groups(T, group):
    _run(1024, 16, group, T)


@pytest.mark.parametrize("N", [1, 8, 17, 127, 129, 700, 2049, 4096])
@pytest.mark.parametrize("T", [1, 20, 50])
def test_odd_output_widths(N, T):
    _run(N, 16, 64, T)


@pytest.mark.parametrize("H,d_h,group", [(1, 128, 128), (1, 128, 32), (3, 128, 64), (5, 128, 32), (20, 128, 128), (7, 64, 64),
                                         (16, 256, 128), (1, 64, 32), (128, 128, 128), (9, 96, 32)])
@pytest.mark.parametrize("T", [1, 12, 70])
def test_inner_widths(H, d_h, group, T):
    """Inner widths that leave a partial chunk of 256, that hold a single group, and long ones."""
    _run(384, H, group, T, d_h=d_h)


@pytest.mark.parametrize("gate", ["channel", "head", "head_topk", "head_binary", "head_ternary"])
@pytest.mark.parametrize("T", [1, 5, 40, 100])
def test_gates(gate, T):
    _run(512, 16, 64, T, gate=gate, topk=3 if gate == "head_topk" else 0)


@pytest.mark.parametrize("gate", [None, "channel", "head", "head_topk", "head_binary", "head_ternary"])
def test_gates_many_tokens(gate):
    _run(384, 16, 64, 290, gate=gate, topk=3 if gate == "head_topk" else 0, seed=1)


@pytest.mark.parametrize("N,H,d_h,T", [(1, 1, 128, 257), (17, 3, 64, 300), (700, 20, 128, 511), (128, 130, 128, 260), (257, 1, 64, 1000)])
def test_many_tokens_odd_sizes(N, H, d_h, T):
    """Widths that leave partial tiles, and an inner width of more than 16384."""
    _run(N, H, 32, T, d_h=d_h, gate="channel")


def test_many_tokens_rows_of_any_magnitude():
    """Token rows and weight rows spread over 2^-50 .. 2^50: each keeps its own relative precision; a row of
    zeros gives zeros, and an infinity or a NaN stays in its own row."""
    N, H, T, group = 130, 4, 300, 32
    model, w4, g = _make(N, H, group)
    K = H * 128
    w4.scales[:] = (w4.scales.float() * torch.exp2(torch.arange(N, device="cuda") % 11 * 10.0 - 50)[:, None]).bfloat16()
    o = torch.randn(T, K, generator=g, device="cuda")
    o = (o * torch.exp2(torch.arange(T, device="cuda") % 7 * 15.0 - 45)[:, None]).bfloat16()
    o[7] = 0
    o[11, 3] = float("inf")
    o[12, 5] = float("nan")
    y = model.gate_out_w4(o, w4).double().cpu()
    model.sync_status()
    W = torch.from_numpy(R.w4_dense(w4.codes.cpu().numpy(), w4.scales.float().cpu().numpy(), group))
    a = o.double().cpu()
    live = [t for t in range(T) if t not in (11, 12)]
    ref, S = a[live] @ W.t(), a[live].abs() @ W.abs().t()
    tol = 2.0 ** -8 * ref.abs() + (2.0 ** -23 * (K / 16 + 64) + 2.0 ** -12) * S
    tol += 2.0 ** -39 * a[live].abs().amax(1, keepdim=True) * W.abs().sum(1)
    assert bool(((y[live] - ref).abs() <= tol).all())
    assert not y[7].any()
    assert not y[11].isfinite().any() and bool(y[12].isnan().all())


def test_every_code_and_position():
    """Each code 0 .. 15 at each place of a word, one at a time: exact."""
    import gated_mla_b200 as gmla
    N, K = 16, 256
    model = gmla.GatedMLA(d_model=N, n_heads=2, d_h=128, d_c=512, weights={})
    code = torch.arange(16).view(16, 1).expand(16, K)
    codes = (code[:, 0::2] | (code[:, 1::2] << 4)).to(torch.uint8).cuda()
    w4 = gmla.W4Weight(codes.contiguous(), torch.ones(N, 2, dtype=torch.bfloat16, device="cuda"), 128)
    for k0 in range(0, K, 64):
        o = torch.zeros(64, K, dtype=torch.bfloat16, device="cuda")
        o[torch.arange(64), k0 + torch.arange(64)] = 1
        y = model.gate_out_w4(o, w4)
        assert torch.equal(y.float(), (torch.arange(16, device="cuda").float() - 8).expand(64, 16))


def test_one_nibble_at_a_time_lands_at_its_column():
    import gated_mla_b200 as gmla
    N, K = 128, 512
    g = torch.Generator().manual_seed(0)
    full = torch.randint(0, 16, (N, K), generator=g)
    codes = (full[:, 0::2] | (full[:, 1::2] << 4)).to(torch.uint8).cuda().contiguous()
    scales = torch.full((N, K // 32), 0.5, dtype=torch.bfloat16, device="cuda")
    model = gmla.GatedMLA(d_model=N, n_heads=4, d_h=128, d_c=512, weights={})
    w4 = gmla.W4Weight(codes, scales, 32)
    eye = torch.eye(K, dtype=torch.bfloat16, device="cuda")
    want = ((full.float() - 8) / 2).t().cuda()
    for step in (8, 64, 512):
        for k in range(0, K, step):
            assert torch.equal(model.gate_out_w4(eye[k:k + step].contiguous(), w4).float(), want[k:k + step])


def test_quantize_w4_rounds_to_the_nearest_code():
    import gated_mla_b200 as gmla
    W = torch.randn(48, 256, device="cuda")
    W[3, :64] = 0
    w4 = gmla.quantize_w4(W, 64)
    back = torch.from_numpy(R.w4_dense(w4.codes.cpu().numpy(), w4.scales.float().cpu().numpy(), 64))
    step = w4.scales.double().cpu().repeat_interleave(64, 1)
    # half a step, and the scale (largest / 7) is itself rounded to bf16: 7 codes of it may be 2^-8 short
    assert bool(((back - W.double().cpu()).abs() <= step * (0.5 + 7 * 2.0 ** -8) + 1e-12).all())
    assert not back[3, :64].any()


def test_a_row_of_y_does_not_depend_on_the_others_and_repeats():
    model, w4, o, z, y = _run(900, 16, 128, 40)
    for _ in range(5):
        assert torch.equal(model.gate_out_w4(o, w4, z), y)
    assert torch.equal(model.gate_out_w4(torch.cat([o[:33], o[:31]]), w4)[:33], y[:33])


def test_streams_graphs_and_refusals():
    import gated_mla_b200 as gmla
    model, w4, o, z, y = _run(512, 16, 64, 6, gate="channel")
    o2 = o.flip(0).contiguous()
    y2 = model.gate_out_w4(o2, w4, z)
    big = o.repeat(20, 1)
    zb = z.repeat(20, 1)
    yb = model.gate_out_w4(big, w4, zb)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        with torch.cuda.stream(s1):
            a, c = model.gate_out_w4(o, w4, z), model.gate_out_w4(big, w4, zb)
        with torch.cuda.stream(s2):
            b = model.gate_out_w4(o2, w4, z)
    torch.cuda.synchronize()
    assert torch.equal(a, y) and torch.equal(b, y2) and torch.equal(c, yb)
    outs, graphs = [torch.empty_like(y), torch.empty_like(yb)], [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for gph, oo, zz, out in zip(graphs, (o, big), (z, zb), outs):
        with torch.cuda.graph(gph):
            model.gate_out_w4(oo, w4, zz, y_out=out)
    for _ in range(20):
        with torch.cuda.stream(s1):
            graphs[0].replay()
        with torch.cuda.stream(s2):
            graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], y) and torch.equal(outs[1], yb)
    assert model.gate_out_w4(o[:0], w4).shape == (0, 512)
    for bad in (lambda: model.gate_out_w4(o.float(), w4), lambda: model.gate_out_w4(o[:, :1024], w4),
                lambda: model.gate_out_w4(o, gmla.W4Weight(w4.codes, w4.scales, 32)),
                lambda: model.gate_out_w4(o, gmla.W4Weight(w4.codes, w4.scales.float(), 64)),
                lambda: model.gate_out_w4(o, gmla.W4Weight(w4.codes[:-1], w4.scales, 64)),
                lambda: model.gate_out_w4(o, w4, z[:, :7]), lambda: model.gate_out_w4(o, w4, z.bfloat16()),
                lambda: model.gate_out_w4(o, gmla.W4Weight(w4.codes, w4.scales, 48))):
        with pytest.raises(ValueError):
            bad()
    f32 = gmla.GatedMLA(d_model=512, n_heads=16, d_h=128, d_c=512, dtype=torch.float32, weights={})
    with pytest.raises(gmla._lib.GmlaError) as e:
        f32.gate_out_w4(o.float(), w4)
    assert e.value.status == gmla._lib.GMLA_ERR_UNSUPPORTED
