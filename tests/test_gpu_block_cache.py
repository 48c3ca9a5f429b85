"""The E4M3 latent cache with one scale for every block of rows: cache_append equals a
sequential append bit for bit (powers of two scale exactly, so every rounding is the
formula's), and decode over it stays within the bound of operators_ref.decode, which counts
each rounding of the path."""
import numpy as np
import pytest
import torch

import operators_ref as R

pytestmark = pytest.mark.gpu
D = 512


def _model(H=16, gate="channel", W_k=None, W_v=None, d_h=128, **kw):
    import gated_mla_b200 as gmla
    weights = {}
    if W_k is not None:
        weights = dict(W_k=W_k, W_v=W_v)
    return gmla.GatedMLA(d_model=256, n_heads=H, d_h=d_h, d_c=D, gate_mode=gate, cache_fp8="block", weights=weights, **kw)


class Pool:
    """A cache on both sides. Codes of rows that nobody owns are NaN, their scales too."""

    def __init__(self, B, cap, page, block, seed=0, extra=3):
        import gated_mla_b200 as gmla
        g = np.random.default_rng(seed)
        self.B, self.page, self.block = B, page, block
        if page:
            M = -(-cap // page)
            self.table = g.permutation(B * M + extra)[:B * M].reshape(B, M).astype(np.int32)
            rows, n = (B * M + extra) * page, (B * M + extra, page // block)
            shape = (B * M + extra, page, D)
        else:
            self.table, rows, shape = None, B * cap, (B, cap, D)
            n = (B, -(-cap // block))
        self.cap = cap
        self.per = n[1]
        self.codes = np.full((rows, D), np.nan)
        self.scales = np.full(n[0] * n[1], np.nan)
        data = torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        sc = torch.full(n, float("nan"), dtype=torch.float32, device="cuda")
        self.cache = gmla.LatentCache(data, None if self.table is None else torch.from_numpy(self.table).cuda(),
                                      scales=sc, scale_block=block)

    def row_of(self, b, p):
        return b * self.cap + p if self.table is None else int(self.table[b, p // self.page]) * self.page + p % self.page

    def block_of(self, b, p):
        return b * self.per + p // self.block if self.table is None else self.row_of(b, p) // self.block

    def append(self, model, latents, new, lens, pad=0):
        """On both sides; `latents` bf16 on the GPU, `pad` rows behind the last sequence's."""
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        x = latents
        if pad:
            x = torch.cat([latents, torch.full((pad, D), float("nan"), dtype=latents.dtype, device="cuda")])
        model.cache_append(x, torch.from_numpy(cu).cuda(), torch.tensor(list(lens), dtype=torch.int32, device="cuda"),
                           self.cache)
        R.append(self.codes, self.scales, self.row_of, self.block_of, latents.double().cpu().numpy(), cu, lens, self.block)

    def same(self):
        got = self.cache.data.view(torch.uint8).cpu().numpy().reshape(-1, D)
        want = np.where(np.isnan(self.codes), 0x7F, R.e4m3_codes(np.nan_to_num(self.codes)))
        assert np.array_equal(got, want)
        assert np.array_equal(self.cache.scales.cpu().numpy().reshape(-1).astype(np.float64), self.scales, equal_nan=True)

    def rows(self, b, L):
        """Rows 0 .. L - 1 of a sequence as values, and their scales."""
        out, s = np.empty((L, D)), np.empty(L)
        for p in range(L):
            s[p] = self.scales[self.block_of(b, p)]
            out[p] = self.codes[self.row_of(b, p)] * s[p]
        return out, s


def _latents(T, seed, spread=1.0, tiny=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, D, generator=g, device="cuda") * torch.exp(spread * torch.randn(T, 1, generator=g, device="cuda"))
    if tiny:      # elements far below their row's largest: E4M3's subnormal range, where rounding again shows
        x = x * torch.exp2(-12 * torch.rand(T, D, generator=g, device="cuda"))
    return x.to(torch.bfloat16)


@pytest.mark.parametrize("page", [0, 8, 64, 128, 256])
@pytest.mark.parametrize("block", [1, 2, 4, 8, 16, 32, 64, 128])
def test_append_equals_the_sequential_append(page, block):
    if page and block > page:
        pytest.skip("a block lies within a page")
    model = _model()
    B, cap = 5, 400 if page else 391
    pool = Pool(B, cap, page, block, seed=block)
    lens = np.zeros(B, int)
    for step, new in enumerate([[0, 1, 130, 5, 64], [3, 0, 1, 1, 64], [1, 1, 1, 1, 1], [0, 0, 0, 0, 0], [140, 7, 2, 16, 129],
                                [1, 250, 17, 1, 1]]):
        lens += new
        x = _latents(int(np.sum(new)), seed=10 * block + step, spread=0.3 + step, tiny=True)
        pool.append(model, x, new, lens.tolist(), pad=step % 3)
        pool.same()
    model.sync_status()


def test_append_of_single_tokens_grows_the_scale_of_a_block():
    model = _model()
    pool = Pool(3, 64, 64, 64)
    for i in range(40):
        x = (_latents(3, seed=i, tiny=True).float() * 2.0 ** (i % 11)).to(torch.bfloat16)
        pool.append(model, x, [1, 1, 1], [i + 1] * 3)
    pool.same()


def test_append_many_short_sequences_and_long_prompts():
    model = _model()
    g = np.random.default_rng(5)
    for block, B, hi in ((16, 1200, 3), (1, 700, 4), (64, 3, 2500)):
        new = g.integers(0, hi + 1, B)
        past = g.integers(0, 40, B)
        pool = Pool(B, 40 + hi, 64, block, seed=B, extra=0)
        pool.append(model, _latents(int(past.sum()), seed=1), past, past.tolist())
        pool.append(model, _latents(int(new.sum()), seed=2), new, (past + new).tolist())
        pool.same()


def test_append_extremes_zeros_and_saturation():
    model = _model()
    pool = Pool(1, 16, 16, 4)
    x = torch.zeros(16, D, dtype=torch.bfloat16, device="cuda")
    x[4, 3] = 448.0                 # exactly 448 * 2^0
    x[5, 3] = 1.0
    x[8, 0] = 450.0                 # the next bf16 above 448: scale 2
    x[12, 0], x[13, 1] = 2.0 ** 60, -1.0     # beyond 448 * 2^32: the largest scale, saturated
    pool.append(model, x, [16], [16])
    pool.same()
    assert pool.cache.scales[int(pool.table[0, 0])].tolist() == [2.0 ** -32, 1.0, 2.0, 2.0 ** 32]


def test_append_strided_rows():
    model = _model()
    pool = Pool(2, 64, 64, 16)
    wide = torch.cat([_latents(50, 3), _latents(50, 4)], 1)
    x = wide[:, 512:]
    pool.append(model, x, [20, 30], [20, 30])
    pool.same()
    model.sync_status()


def test_append_out_of_range_is_skipped_and_reported():
    import gated_mla_b200 as gmla
    for what in ("page", "length", "past"):
        model = _model()
        pool = Pool(3, 32, 16, 16)
        before = pool.cache.data.view(torch.uint8).clone()
        lens = [4, 4, 4]
        if what == "page":
            pool.cache.block_table[1, 0] = 10 ** 6
        elif what == "length":
            lens[1] = 33
        else:
            lens[1] = 2
        cu = torch.tensor([0, 4, 8, 12], dtype=torch.int32, device="cuda")
        x = _latents(12, 1)
        model.cache_append(x, cu, torch.tensor(lens, dtype=torch.int32, device="cuda"), pool.cache)
        with pytest.raises(gmla._lib.GmlaError) as e:
            model.sync_status()
        assert e.value.status == gmla._lib.GMLA_ERR_DEVICE_RANGE
        now = pool.cache.data.view(torch.uint8).view(-1, 16, D)
        changed = (now != before.view(-1, 16, D)).flatten(1).any(1)
        want = torch.zeros_like(changed)
        want[[int(pool.table[0, 0]), int(pool.table[2, 0])]] = True
        assert torch.equal(changed, want), what


def test_append_of_fewer_rows_than_the_offsets_name_is_reported():
    import gated_mla_b200 as gmla
    model = _model()
    pool = Pool(2, 64, 16, 16)
    x = _latents(6, 1)
    model.cache_append(x, torch.tensor([0, 4, 9], dtype=torch.int32, device="cuda"),
                       torch.tensor([4, 5], dtype=torch.int32, device="cuda"), pool.cache)
    with pytest.raises(gmla._lib.GmlaError) as e:
        model.sync_status()
    assert e.value.status == gmla._lib.GMLA_ERR_DEVICE_RANGE


# ---------------------------------------------------------------------------
def _attend(H, lens, page, block, gate="channel", seed=0, q_mul=1.0, spread=1.0, d_h=128, cap=None, plant=None, topk=0,
            seqs=None, logits=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    B = len(lens)
    W_k, W_v = (n(H, d_h, D) / D ** 0.5).to(torch.bfloat16), (n(H, d_h, D) / D ** 0.5).to(torch.bfloat16)
    model = _model(H, gate, W_k, W_v, d_h=d_h, gate_topk=topk)
    pool = Pool(B, cap or max(max(lens), 1), page, block, seed=seed)
    x = _latents(sum(lens), seed + 1, spread)
    q = (q_mul * n(B, H, d_h)).to(torch.bfloat16)
    if plant:
        x = plant(x, q, W_k)
    pool.append(model, x, lens, lens)
    z = 1.4 * n(B, H * d_h if gate == "channel" else H) if logits else None
    L = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o = model.decode(q, z, pool.cache, L)
    model.sync_status()
    assert o.isfinite().all()
    wk, wv, qq = (t.double().cpu().numpy() for t in (W_k, W_v, q))
    got = o.double().cpu().numpy().reshape(B, H, d_h)
    gv = (R.gate_values(z.double().cpu().numpy(), gate, H, d_h, topk).reshape(B, H, d_h) if logits else np.ones((B, H, d_h)))
    num = den = 0.0
    for b in range(B) if seqs is None else seqs:
        c, sc = pool.rows(b, lens[b])
        ref, bound = R.decode(qq[b], c, wk, wv, 1 / np.sqrt(d_h), sc)
        # the gate: a fast exponential and reciprocal, 2^-20 of the value
        assert np.all(np.abs(got[b] - gv[b] * ref) <= gv[b] * (bound + 2.0 ** -20 * np.abs(ref)) + 1e-30), b
        num += ((got[b] - gv[b] * ref) ** 2).sum()
        den += ((gv[b] * ref) ** 2).sum()
    if den:
        assert (num / den) ** 0.5 <= 1e-2      # the framework's bound for a bf16 path
    return model, pool, q, z, L, o


@pytest.mark.parametrize("block", [1, 16, 64, 128])
def test_decode_16_heads_contiguous(block):
    _attend(16, [1, 127, 128, 129, 0, 700, 2, 64], 0, block, seed=block, cap=719)


@pytest.mark.parametrize("page,block", [(8, 1), (8, 8), (16, 4), (64, 64), (128, 16), (128, 128), (256, 32), (384, 128)])
def test_decode_32_heads_paged(page, block):
    _attend(32, [1, 63, 64, 65, 0, 900, 257], page, block, gate="head", seed=page + block)


def test_decode_head_counts_and_head_dims():
    for H, d_h, gate in ((1, 128, "head"), (5, 128, "channel"), (24, 128, "head"), (64, 128, "channel"), (16, 256, "channel"),
                         (128, 128, "head")):
        _attend(H, [300, 17], 64, 32, gate=gate, seed=H, d_h=d_h)


@pytest.mark.parametrize("gate", ["head_topk", "head_binary", "head_ternary"])
def test_decode_hard_gates(gate):
    _attend(32, [130, 400, 9], 64, 64, gate=gate, seed=7, topk=6 if gate == "head_topk" else 0)


def test_decode_ungated():
    _attend(16, [200, 31], 64, 16, seed=9, logits=False)


def test_decode_scales_far_apart():
    """Rows whose sizes differ by factors of thousands: the reference of the softmax follows score and scale together."""
    _attend(16, [1500, 260], 64, 1, seed=3, spread=3.0, q_mul=0.02)


def test_decode_long_context_under_one_dominant_token():
    """One token takes half of the softmax, 30000 others share the rest: their weights, each about
    2^-16 of the largest, must survive the 8-bit products."""
    L = 30000

    def plant(x, q, W_k):
        qa = torch.einsum("hd,hdc->hc", q[0].float(), W_k.float())
        sink = torch.linalg.lstsq(qa[:16], torch.full((16, 1), 11.0 * 128 ** 0.5, device="cuda")).solution[:, 0]
        x = x.clone()
        x[0] = sink.to(torch.bfloat16)
        return x
    _attend(16, [L], 64, 64, seed=21, spread=0.1, q_mul=0.3, plant=plant)


def test_decode_peaked_scores_rescale():
    _attend(16, [900, 1300], 64, 64, seed=4, q_mul=6.0, spread=0.5)


def test_decode_many_segments_sampled():
    _attend(16, [20000, 3, 700], 128, 128, seed=8, spread=0.5)


def test_decode_bad_scale_and_page_are_reported():
    import gated_mla_b200 as gmla
    for what in ("nan", "zero", "huge", "page"):
        model, pool, q, z, L, _ = _attend(16, [100, 50], 64, 64, seed=2)
        if what == "page":
            pool.cache.block_table[0, 1] = 10 ** 6
        else:
            pool.cache.scales[int(pool.table[0, 0]), 0] = {"nan": float("nan"), "zero": 0.0, "huge": 2.0 ** 40}[what]
        o2 = model.decode(q, z, pool.cache, L)
        with pytest.raises(gmla._lib.GmlaError) as e:
            model.sync_status()
        assert e.value.status == gmla._lib.GMLA_ERR_DEVICE_RANGE, what
        assert o2[1].isfinite().all()


def test_context_parallel_shares_merge_to_the_whole():
    from gated_mla_b200 import _lib as lib
    model, pool, q, z, L, o = _attend(16, [700, 130, 300], 64, 32, seed=13)
    B, H = 3, 16
    parts = []
    for lo, hi in (([0, 0, 0], [256, 0, 300]), ([256, 0, 0], [700, 130, 0])):
        part = torch.empty(B, H, D + 4, device="cuda")
        nb = lib.gmla_decode_workspace_size(model.cfg, B)
        ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
        s, e = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in (lo, hi))
        lib.check(lib.gmla_decode_partial(model.cfg, model.w, q.data_ptr(), z.data_ptr(), pool.cache.struct(), s.data_ptr(),
                                          e.data_ptr(), B, part.data_ptr(), ws.data_ptr(), nb,
                                          torch.cuda.current_stream().cuda_stream), "partial")
        parts.append(part)
    both = torch.stack(parts)
    out = torch.empty_like(o)
    nb = lib.gmla_decode_merge_workspace_size(model.cfg, B)
    ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
    lib.check(lib.gmla_decode_merge(model.cfg, model.w, both.data_ptr(), 2, z.data_ptr(), B, out.data_ptr(), ws.data_ptr(),
                                    nb, torch.cuda.current_stream().cuda_stream), "merge")
    # both are within half of the framework's relative bound of the same values
    assert float((out.float() - o.float()).norm() / o.float().norm()) < 1e-2


def test_cache_beyond_4_gb():
    """Rows, codes and scales past 2^32 bytes: the last pages of a 4.8 GB pool."""
    import gated_mla_b200 as gmla
    page, block, n_pages = 128, 1, 73500
    data = torch.empty(n_pages, page, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scales = torch.empty(n_pages, page, device="cuda")
    table = torch.tensor([[n_pages - 1, n_pages - 2]], dtype=torch.int32, device="cuda")
    cache = gmla.LatentCache(data, table, scales=scales)
    small = gmla.LatentCache(torch.empty(2, page, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
                             torch.tensor([[1, 0]], dtype=torch.int32, device="cuda"), scales=torch.empty(2, page, device="cuda"))
    g = torch.Generator(device="cuda").manual_seed(1)
    W = (torch.randn(2, 16, 128, D, generator=g, device="cuda") / D ** 0.5).to(torch.bfloat16)
    model = _model(16, "channel", W[0].contiguous(), W[1].contiguous())
    x = _latents(200, 1)
    cu, L = torch.tensor([0, 200], dtype=torch.int32, device="cuda"), torch.tensor([200], dtype=torch.int32, device="cuda")
    q = torch.randn(1, 16, 128, generator=g, device="cuda").to(torch.bfloat16)
    outs = []
    for c in (cache, small):
        model.cache_append(x, cu, L, c)
        outs.append(model.decode(q, None, c, L))
    model.sync_status()
    a, b = data[-2:].view(torch.uint8), small.data.view(torch.uint8)
    assert torch.equal(a[1], b[1]) and torch.equal(a[0, :72], b[0, :72])
    assert torch.equal(scales[-1], small.scales[1]) and torch.equal(scales[-2, :72], small.scales[0, :72])
    assert torch.equal(outs[0], outs[1])


def test_two_streams_and_two_graphs_do_not_share_scratch():
    """Decodes of one layer on two streams, and two captured graphs replayed side by side."""
    model, pool, q, z, L, o = _attend(16, [1500, 130, 900, 333], 64, 32, seed=31)
    q2 = q.flip(0).contiguous()
    want2 = model.decode(q2, z, pool.cache, L)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        with torch.cuda.stream(s1):
            a = model.decode(q, z, pool.cache, L)
        with torch.cuda.stream(s2):
            b = model.decode(q2, z, pool.cache, L)
    torch.cuda.synchronize()
    assert torch.equal(a, o) and torch.equal(b, want2)
    outs, graphs = [torch.empty_like(o), torch.empty_like(o)], [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for gph, qq, out in zip(graphs, (q, q2), outs):
        with torch.cuda.graph(gph):
            model.decode(qq, z, pool.cache, L, o_out=out)
    for _ in range(20):
        with torch.cuda.stream(s1):
            graphs[0].replay()
        with torch.cuda.stream(s2):
            graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], o) and torch.equal(outs[1], want2)
    model.sync_status()


def test_what_a_block_scaled_layer_refuses():
    import gated_mla_b200 as gmla
    model, pool, q, z, L, o = _attend(16, [40], 64, 32, seed=1)
    plain = gmla.LatentCache(pool.cache.data, pool.cache.block_table)
    x = _latents(4, 1)
    cu = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        model.cache_append(x, cu, L, plain)
    with pytest.raises(gmla._lib.GmlaError):
        model.decode(q, z, plain, L)
    with pytest.raises(ValueError):
        model.latent_project(x, L, L, pool.cache)
    with pytest.raises(ValueError):
        model.cache_append(x.float(), cu, L, pool.cache)
    with pytest.raises(ValueError):
        gmla.LatentCache(pool.cache.data, pool.cache.block_table, scales=pool.cache.scales, scale_block=16).struct()
    with pytest.raises(gmla._lib.GmlaError):
        model.prefill(q, z, pool.cache, cu, 4)
