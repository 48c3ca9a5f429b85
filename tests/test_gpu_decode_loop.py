"""The operators of a serving step used together: plan_batch, add_rms_norm, the projection
with cache_append, decode over the block-scaled cache and the 4-bit output product, over
prompts and several single-token steps. Every stage is held against 64 bits on what the stage
before it gave; the same steps captured once and replayed give the same bits."""
import numpy as np
import pytest
import torch

import operators_ref as R

pytestmark = pytest.mark.gpu
N, H, DH, D, PAGE, BLOCK, GROUP, M = 512, 16, 128, 512, 64, 32, 64, 6
PROMPTS = [1, 63, 64, 200, 0]        # the last slot of the batch stays idle
B = len(PROMPTS)
BF16 = 2.0 ** -8                     # half a step, relative


class Server:
    def __init__(self, seed=0):
        import gated_mla_b200 as gmla
        self.gmla = gmla
        g = torch.Generator(device="cuda").manual_seed(seed)
        n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        w = dict(W_q=n(H * DH, N) / N ** 0.5, W_c=n(D, N) / N ** 0.5, W_g=n(H * DH, N) / N ** 0.5,
                 W_k=n(H, DH, D) / D ** 0.5, W_v=n(H, DH, D) / D ** 0.5)
        self.w = {k: v.to(torch.bfloat16) for k, v in w.items()}
        self.layer = gmla.GatedMLA(d_model=N, n_heads=H, d_h=DH, d_c=D, cache_fp8="block", weights=self.w)
        self.w4 = gmla.quantize_w4(n(N, H * DH) / (H * DH) ** 0.5, GROUP)
        self.norm_w = (1 + 0.1 * n(N)).to(torch.bfloat16)
        pages = B * M + 2
        self.table = torch.full((B, M), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        self.cache = gmla.LatentCache(
            torch.full((pages, PAGE, D), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn), self.table,
            scales=torch.full((pages, PAGE // BLOCK), float("nan"), device="cuda"), scale_block=BLOCK)
        self.cached = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.g = g

    def prefill(self):
        new = torch.tensor(PROMPTS, dtype=torch.int32, device="cuda")
        T = sum(PROMPTS) + 3
        x = torch.randn(T, N, generator=self.g, device="cuda").to(torch.bfloat16)
        plan = self.gmla.plan_batch(self.cached, new, self.table, self.free, PAGE, T)
        nr = self.gmla.add_rms_norm(x, self.norm_w)
        self.layer.latent_project(nr.out, plan.positions, plan.seq_ids, self.cache, cu_seqlens=plan.cu_seqlens,
                                  seq_lens=plan.seq_lens)
        self.cached.copy_(plan.seq_lens)
        self.used = int(plan.pages_used)
        return x, plan, nr

    def step(self, x, h, new, free):
        """One token for every live sequence; x [B, N] the branch, h [B, N] the residual stream."""
        plan = self.gmla.plan_batch(self.cached, new, self.table, free, PAGE, B)
        nr = self.gmla.add_rms_norm(x, self.norm_w, h)
        q, z = self.layer.latent_project(nr.out, plan.positions, plan.seq_ids, self.cache, cu_seqlens=plan.cu_seqlens,
                                         seq_lens=plan.seq_lens)
        o = self.layer.decode(q, z, self.cache, plan.seq_lens)
        y = self.layer.gate_out_w4(o, self.w4)
        return plan, nr, q, z, o, y


def _np(t):
    return t.double().cpu().numpy()


def _check_norm(nr, x, w, h=None):
    s = _np(x) + (_np(h) if h is not None else 0)
    ref = s / np.sqrt((s ** 2).mean(1, keepdims=True) + 1e-6) * _np(w)
    # bf16 output, and the fp32 sum of N squares, its root and two products (2^-24 (N + 8))
    assert np.all(np.abs(_np(nr.out) - ref) <= np.abs(ref) * (BF16 + 2.0 ** -24 * (N + 8)))
    if h is not None:
        assert np.all(np.abs(_np(nr.residual) - s) <= np.abs(s) * BF16 * (1 + 2.0 ** -10))


def _check_cache_rows(srv, table, xn, spans):
    """Rows (sequence, first position, first token row, count) hold W_c x, rounded to bf16 and then to
    E4M3 under their block's scale: 2^-8 and 2^-4 of the value, or half the subnormal step, 2^-10 scale,
    below that; fp32 sums over N terms. A scale that grew rounded the subnormal part again, under
    scales that halve: twice that half step in all."""
    W = _np(srv.w["W_c"])
    codes, scales = srv.cache.data.view(torch.uint8).cpu().numpy(), _np(srv.cache.scales)
    for b, p0, t0, n in spans:
        ref = xn[t0:t0 + n] @ W.T
        mag = np.abs(xn[t0:t0 + n]) @ np.abs(W.T)
        for i in range(n):
            page, at = table[b, (p0 + i) // PAGE], (p0 + i) % PAGE
            s = scales[page, at // BLOCK]
            got = R.e4m3_values(codes[page, at]) * s
            lat = np.abs(ref[i]) * (1 + BF16) + 2.0 ** -23 * N * mag[i]
            tol = 2.0 ** -23 * N * mag[i] + BF16 * np.abs(ref[i]) + 2.0 ** -4 * lat + 2 * 2.0 ** -10 * s
            assert np.all(np.abs(got - ref[i]) <= tol), (b, p0 + i)


def _cache_rows(srv, table, b, L):
    codes, scales = srv.cache.data.view(torch.uint8).cpu().numpy(), _np(srv.cache.scales)
    s = np.array([scales[table[b, p // PAGE], p % PAGE // BLOCK] for p in range(L)])
    c = np.array([R.e4m3_values(codes[table[b, p // PAGE], p % PAGE]) for p in range(L)]).reshape(L, D)
    return c * s[:, None], s


def _check_plan(plan, want):
    for k in ("seq_lens", "cu_seqlens", "positions", "seq_ids", "slots"):
        assert np.array_equal(getattr(plan, k).cpu().numpy(), want[k]), k
    assert int(plan.pages_used) == want["pages_used"]


def test_prompts_then_steps_stage_by_stage():
    srv = Server()
    free = srv.free.cpu().numpy()
    want = R.plan([0] * B, PROMPTS, srv.table.cpu().numpy(), free, PAGE, sum(PROMPTS) + 3)
    x, plan, nr = srv.prefill()
    srv.gmla.sync_status()
    srv.layer.sync_status()
    _check_plan(plan, want)
    assert np.array_equal(srv.table.cpu().numpy(), want["table"])
    _check_norm(nr, x, srv.norm_w)
    cu = want["cu_seqlens"]
    _check_cache_rows(srv, want["table"], _np(nr.out), [(b, 0, cu[b], PROMPTS[b]) for b in range(B)])

    new = torch.tensor([1, 1, 1, 1, 0], dtype=torch.int32, device="cuda")
    h = torch.randn(B, N, generator=srv.g, device="cuda").to(torch.bfloat16)
    y = torch.randn(B, N, generator=srv.g, device="cuda").to(torch.bfloat16)
    table, lens, used = want["table"], list(PROMPTS), want["pages_used"]
    wk, wv, Wq, Wg = (_np(srv.w[k]) for k in ("W_k", "W_v", "W_q", "W_g"))
    W4 = R.w4_dense(srv.w4.codes.cpu().numpy(), srv.w4.scales.float().cpu().numpy(), GROUP)
    w4s = np.repeat(_np(srv.w4.scales), GROUP, axis=1)
    K = H * DH
    for _ in range(3):
        x, h_in = y, h
        want = R.plan(lens, [1, 1, 1, 1, 0], table, free[used:], PAGE, B)
        plan, nr, q, z, o, y = srv.step(x, h_in, new, srv.free[used:].contiguous())
        srv.gmla.sync_status()
        srv.layer.sync_status()
        _check_plan(plan, want)
        table, lens, used = want["table"], want["seq_lens"].tolist(), used + want["pages_used"]
        assert np.array_equal(srv.table.cpu().numpy(), table)
        _check_norm(nr, x, srv.norm_w, h_in)
        xn = _np(nr.out)
        _check_cache_rows(srv, table, xn, [(b, lens[b] - 1, b, 1) for b in range(B - 1)])
        # projections: fp32 sums over N terms, the query rounded to bf16
        for got, W, r in ((_np(q).reshape(B, K), Wq, BF16), (_np(z), Wg, 0.0)):
            ref = xn @ W.T
            tol = r * np.abs(ref) + 2.0 ** -23 * N * (np.abs(xn) @ np.abs(W.T))
            assert np.all(np.abs(got - ref) <= tol * (1 + BF16))
        gv = R.gate_values(_np(z), "channel", H, DH).reshape(B, H, DH)
        got = _np(o).reshape(B, H, DH)
        for b in range(B):
            c, s = _cache_rows(srv, table, b, lens[b])
            ref, bound = R.decode(_np(q)[b].reshape(H, DH), c, wk, wv, 1 / np.sqrt(DH), s)
            assert np.all(np.abs(got[b] - gv[b] * ref) <= gv[b] * (bound + 2.0 ** -20 * np.abs(ref)) + 1e-30), b
        assert not got[B - 1].any() and not _np(y)[B - 1].any()      # the idle slot
        a = _np(o)
        ref, S = a @ W4.T, np.abs(a) @ np.abs(W4.T)
        tol = BF16 * np.abs(ref) + 2.0 ** -23 * ((K / 16 + 64) * S + 12 * 144 * (np.abs(a) @ w4s.T))
        assert np.all(np.abs(_np(y) - ref) <= tol)
        h = nr.residual
        srv.cached.copy_(plan.seq_lens)
        new = torch.tensor([1, 1, 1, 1, 0], dtype=torch.int32, device="cuda")


def test_captured_steps_replay_the_eager_ones():
    """One captured step, replayed: positions, pages, cache, outputs as the eager steps leave them."""
    eager, graph = Server(1), Server(1)
    for s in (eager, graph):
        s.prefill()
    new = torch.tensor([1, 1, 1, 1, 0], dtype=torch.int32, device="cuda")
    x0, h0 = (torch.randn(B, N, generator=eager.g, device="cuda").to(torch.bfloat16) for _ in range(2))
    free = eager.free[eager.used:].contiguous()

    def advance(s, x, h, free):
        plan, nr, _, _, _, y = s.step(x, h, new, free)
        s.cached.copy_(plan.seq_lens)
        x.copy_(y)
        h.copy_(nr.residual)
        k = plan.pages_used.long()
        free.copy_(free[(torch.arange(free.numel(), device="cuda") + k).clamp(max=free.numel() - 1)])

    xs, hs, fs = [x0.clone(), x0.clone()], [h0.clone(), h0.clone()], [free.clone(), free.clone()]
    warm = Server(2)
    warm.prefill()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):      # library handles and kernels are set up outside the capture
        advance(warm, x0.clone(), h0.clone(), warm.free[warm.used:].clone())
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    cap = torch.cuda.CUDAGraph()
    with torch.cuda.graph(cap):
        advance(graph, xs[1], hs[1], fs[1])
    for i in range(70):                # past the end of a page for every sequence
        advance(eager, xs[0], hs[0], fs[0])
        cap.replay()
        if i % 23 == 0:
            assert torch.equal(xs[0], xs[1]) and torch.equal(hs[0], hs[1])
    torch.cuda.synchronize()
    eager.layer.sync_status()
    graph.layer.sync_status()
    eager.gmla.sync_status()
    assert torch.equal(xs[0], xs[1]) and torch.equal(hs[0], hs[1]) and torch.equal(fs[0], fs[1])
    assert torch.equal(eager.table, graph.table) and torch.equal(eager.cached, graph.cached)
    assert torch.equal(eager.cache.data.view(torch.uint8), graph.cache.data.view(torch.uint8))
    assert torch.equal(eager.cache.scales.view(torch.int32), graph.cache.scales.view(torch.int32))
    assert eager.cached.tolist() == [n + 70 if n else 0 for n in PROMPTS]
    assert bool(xs[0].isfinite().all())
