"""The operators around a decode step and their plain forms, for timing.

A serving step of a Gated MLA layer is: plan the batch (block table, positions,
slots), add the residual and normalise, project, append the latents to an 8-bit
cache, attend over that cache, and multiply the gated heads with a 4-bit W_o.
This file names cases of the five operators beside the projection, makes their
inputs, and runs them either through ``gated_mla_b200`` (``own``) or as
elementary torch operations in 32 bits.
"""
import math

import torch

own = False

D_C = 512       # latent width of the tensor-core decode
D_H = 128       # head dim
E4M3_MAX = 448.0
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # the paged decode batch: 64 sequences, one new token each
        dict(name="plan decode b64", op="plan", batch=64, page=64, cached_lo=256, cached_hi=32767, new_lo=1, new_hi=1,
             pad=0),
        # a large mixed step: prompt chunks and decodes in one ragged batch, small pages, padded token rows
        dict(name="plan mixed b999", op="plan", batch=999, page=16, cached_lo=0, cached_hi=4096, new_lo=1, new_hi=257,
             pad=129),
        # a decode step of 8 tokens at d_model 7168, with codes for an 8-bit product
        dict(name="norm t8 d7168 e4m3", op="norm", tokens=8, d=7168, dtype="bf16", group=128, residual=True, out=True),
        # the batch-4 prefill of 4096 tokens each at d_model 7168
        dict(name="norm t16384 d7168", op="norm", tokens=16384, d=7168, dtype="bf16", group=0, residual=True, out=True),
        # one new latent a sequence into a paged cache (64-token pages and scale blocks)
        dict(name="append b64", op="append", batch=64, page=64, block=64, cached_lo=255, cached_hi=4095, new_lo=1,
             new_hi=1),
        # whole prompts into the cache, ragged, with a scale for every 16 tokens
        dict(name="append prompts b7", op="append", batch=7, page=128, block=16, cached_lo=0, cached_hi=99,
             new_lo=1500, new_hi=4096),
        # one short sequence: the latency of a single request's decode
        dict(name="attend b1 short", op="attend", batch=1, heads=16, page=64, block=64, len_lo=200, len_hi=300,
             gate="channel"),
        # the ragged paged decode with per-head gates
        dict(name="attend b64 paged", op="attend", batch=64, heads=32, page=64, block=64, len_lo=256, len_hi=32768,
             gate="head"),
        # long contexts with all 128 heads
        dict(name="attend b8 128k", op="attend", batch=8, heads=128, page=128, block=128, len_lo=131072,
             len_hi=131072, gate="channel"),
        # one token through the largest W_o (128 heads of 128 into d_model 7168)
        dict(name="w4 t1 7168x16384", op="w4", tokens=1, n=7168, heads=128, group=128, gate="none"),
        # the paged decode batch's W_o with the gate still to be applied
        dict(name="w4 t64 4096x4096", op="w4", tokens=64, n=4096, heads=32, group=64, gate="head"),
        # a prompt chunk through the prefill's W_o
        dict(name="w4 t2000 7168x8192", op="w4", tokens=2000, n=7168, heads=64, group=128, gate="channel"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "norm", "append", "attend", "w4"])
    if op == "plan":
        new_hi = rng.choice([1, 1, 2, 64, 300])
        return dict(op=op, batch=_log(rng, 1, 999), page=rng.choice([8, 16, 64, 128, 256]), cached_lo=rng.choice([0, 1, 500]),
                    cached_hi=_log(rng, 600, 4096), new_lo=rng.choice([0, 1]) if new_hi > 1 else 1, new_hi=new_hi,
                    pad=rng.choice([0, 1, 100]))
    if op == "norm":
        d = _log(rng, 96, 8192)
        return dict(op=op, tokens=_log(rng, 1, 12000), d=d if rng.random() < 0.3 else max(128, d // 64 * 64),
                    dtype=rng.choice(["bf16", "bf16", "fp32"]), group=rng.choice([0, 0, 32, 64, 128]),
                    residual=rng.random() < 0.7, out=True)
    if op == "append":
        page = rng.choice([16, 64, 128, 256])
        new_hi = rng.choice([1, 1, 5, 700])
        return dict(op=op, batch=_log(rng, 1, 40), page=page, block=rng.choice([b for b in (1, 8, 16, 64, 128) if b <= page]),
                    cached_lo=rng.choice([0, 1]), cached_hi=_log(rng, 2, 2500), new_lo=1, new_hi=new_hi)
    if op == "attend":
        page = rng.choice([16, 64, 128, 256])
        batch = _log(rng, 1, 48)
        hi = _log(rng, 40, 600000 // batch if batch > 5 else 100000)
        return dict(op=op, batch=batch, heads=rng.choice([16, 16, 24, 32, 64]), page=page,
                    block=rng.choice([b for b in (1, 16, 64, 128) if b <= page]), len_lo=max(1, hi // rng.choice([2, 50])),
                    len_hi=hi, gate=rng.choice(["channel", "head"]))
    heads = rng.choice([16, 20, 32, 64, 128])
    n = _log(rng, 700, 7168)
    return dict(op=op, tokens=_log(rng, 1, 1500), n=n if rng.random() < 0.3 else n // 128 * 128 + 128, heads=heads,
                group=rng.choice([32, 64, 128]), gate=rng.choice(["none", "head", "channel"]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _spread(n, lo, hi, g, log=False):
    """n whole numbers spread evenly over [lo, hi] (over their logarithm), in an order of the seed's: the sum is the case's own."""
    u = (torch.arange(n, dtype=torch.float64) + 0.5) / n
    v = torch.exp(math.log(lo) + u * math.log((hi + 1) / lo)) if log else lo + u * (hi - lo + 1)
    return torch.floor(v).long().clamp(lo, hi)[torch.randperm(n, generator=g)]


def _lengths(case, g):
    """Past and new lengths of each sequence."""
    return (_spread(case["batch"], case["cached_lo"], case["cached_hi"], g),
            _spread(case["batch"], case["new_lo"], case["new_hi"], g))


def _pool_pages(tokens, batch, page):
    """Pages of a pool that holds `tokens` rows of `batch` sequences however they are divided."""
    return int(tokens) // page + batch


def _table(pages, pool, g, width):
    """A block table over a shuffled pool (pages[b] entries a row, the rest -1), and the ids that it leaves free."""
    total = int(pages.sum())
    perm = torch.randperm(pool, generator=g)
    table = torch.full((len(pages), width), -1, dtype=torch.int64)
    table[torch.arange(width)[None, :] < pages[:, None]] = perm[:total]
    return table.int().cuda(), perm[total:].int().cuda()


def _e4m3(v):
    return v.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _plan_inputs(case, g):
    cached, new = _lengths(case, g)
    page = case["page"]
    pool = _pool_pages((cached + new).sum(), case["batch"], page) + 17
    width = -(-(case["cached_hi"] + case["new_hi"]) // page) + 3
    table, free = _table(-(-cached // page), pool, g, width)
    return dict(cached=cached.int().cuda(), new=new.int().cuda(), table=table, free=free, page=page,
                tokens=int(new.sum()) + case["pad"])


def _latent_rows(shape, g):
    """Latents as a layer makes them: Gaussian, with a magnitude of each token's own."""
    rows = torch.randn(*shape, D_C, generator=g, device="cuda")
    return rows * torch.exp(0.5 * torch.randn(*shape, 1, generator=g, device="cuda"))


def _quantised_pool(n_pages, page, block, g):
    """A pool of E4M3 rows with one power-of-two scale for each `block` rows."""
    codes = torch.empty(n_pages, page, D_C, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty(n_pages, page // block, dtype=torch.float32, device="cuda")
    step = max(1, (1 << 17) // page)
    for i in range(0, n_pages, step):
        n = min(step, n_pages - i)
        rows = _latent_rows((n, page), g).view(n, page // block, block * D_C)
        m, e = torch.frexp(rows.abs().amax(-1) / E4M3_MAX)
        s = torch.ldexp(torch.ones_like(m), e - (m == 0.5).int())
        codes[i:i + n] = _e4m3(rows / s[..., None]).view(n, page, D_C)
        scales[i:i + n] = s
    return codes, scales


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    gg = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(case=case)
    op = case["op"]
    if op == "plan":
        st.update(_plan_inputs(case, g))
    elif op == "norm":
        t, d, dt = case["tokens"], case["d"], torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        st["x"] = torch.randn(t, d, generator=gg, device="cuda").to(dt)
        st["residual"] = (4 * torch.randn(t, d, generator=gg, device="cuda")).to(dt) if case["residual"] else None
        st["weight"] = (1 + 0.2 * torch.randn(d, generator=gg, device="cuda")).to(dt)
    elif op == "append":
        cached, new = _lengths(case, g)
        pool, width = _pool_pages((cached + new).sum(), case["batch"], case["page"]), -(-(case["cached_hi"] + case["new_hi"]) // case["page"])
        st["table"], _ = _table(-(-(cached + new) // case["page"]), pool, g, width)
        st["codes"], st["scales"] = _quantised_pool(pool, case["page"], case["block"], gg)
        st["cu"] = torch.cat([torch.zeros(1, dtype=torch.int64), new.cumsum(0)]).int().cuda()
        st["lens"] = (cached + new).int().cuda()
        st["latents"] = _latent_rows((int(new.sum()),), gg).to(torch.bfloat16)
    elif op == "attend":
        B, H, lo, hi = case["batch"], case["heads"], case["len_lo"], case["len_hi"]
        lens = _spread(B, lo, hi, g, log=True)
        pool = _pool_pages(lens.sum(), B, case["page"])
        st["table"], _ = _table(-(-lens // case["page"]), pool, g, -(-hi // case["page"]))
        st["codes"], st["scales"] = _quantised_pool(pool, case["page"], case["block"], gg)
        st["lens"], st["max_len"] = lens.int().cuda(), int(lens.max())
        st["q"] = torch.randn(B, H, D_H, generator=gg, device="cuda").to(torch.bfloat16)
        width = H * D_H if case["gate"] == "channel" else H
        st["gate"] = 1.4 * torch.randn(B, width, generator=gg, device="cuda")
        w = torch.randn(2, H, D_H, D_C, generator=gg, device="cuda") / math.sqrt(D_C)
        st["W_k"], st["W_v"] = w.to(torch.bfloat16)
    else:
        t, n, k, group = case["tokens"], case["n"], case["heads"] * D_H, case["group"]
        w = (torch.randn(n, k, generator=gg, device="cuda") / math.sqrt(k)).view(n, k // group, group)
        s = (w.abs().amax(-1) / 7).to(torch.bfloat16)
        code = (torch.round(w / s.float()[..., None]).clamp(-8, 7) + 8).to(torch.uint8).view(n, k)
        st["codes"], st["scales"] = code[:, 0::2] | (code[:, 1::2] << 4), s
        st["o"] = torch.randn(t, k, generator=gg, device="cuda").to(torch.bfloat16)
        width = {"none": 0, "head": case["heads"], "channel": k}[case["gate"]]
        st["gate"] = 1.4 * torch.randn(t, width, generator=gg, device="cuda") if width else None
    return st


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _plan_plain(st):
    cached, new, page, T = st["cached"], st["new"], st["page"], st["tokens"]
    zero = torch.zeros(1, dtype=torch.int32, device=cached.device)
    lens = cached + new
    cu = torch.cat([zero, torch.cumsum(new, 0, dtype=torch.int32)])
    have, need = (cached + page - 1) // page, (lens + page - 1) // page
    first = torch.cumsum(need - have, 0, dtype=torch.int32) - (need - have)
    j = torch.arange(st["table"].shape[1], dtype=torch.int32, device=cached.device)[None, :]
    fresh = (j >= have[:, None]) & (j < need[:, None])
    pick = torch.where(fresh, first[:, None] + j - have[:, None], 0).long()
    st["table"].copy_(torch.where(fresh, st["free"][pick], st["table"]))
    t = torch.arange(T, dtype=torch.int32, device=cached.device)
    seq = torch.searchsorted(cu[1:], t, right=True).clamp(max=len(cached) - 1)
    live = t < cu[-1]
    pos = cached[seq] + t - cu[seq]
    entry = st["table"][seq, (pos // page).clamp(0, st["table"].shape[1] - 1).long()].long()
    none = torch.full_like(t, -1)
    return dict(block_table=st["table"], seq_lens=lens, cu_seqlens=cu, positions=torch.where(live, pos, none),
                seq_ids=torch.where(live, seq.int(), none), slots=torch.where(live, entry * page + pos % page, none.long()),
                pages_used=(need - have).sum(dtype=torch.int32).view(1))


def _norm_plain(st):
    case = st["case"]
    x = st["x"].float()
    s = x + st["residual"].float() if case["residual"] else x
    y = s * torch.rsqrt(s.square().mean(-1, keepdim=True) + EPS) * st["weight"].float()
    got = dict(out=y.to(st["x"].dtype))
    if case["residual"]:
        got["residual"] = s.to(st["x"].dtype)
    if case["group"]:
        t, d, group = case["tokens"], case["d"], case["group"]
        n = -(-d // group)
        yg = torch.nn.functional.pad(y, (0, n * group - d)).view(t, n, group)
        top = yg.abs().amax(-1)
        scale = torch.where(top > 0, top / E4M3_MAX, torch.ones_like(top))
        got["codes"] = _e4m3(yg / scale[..., None]).view(t, n * group)[:, :d]
        got["scales"] = scale
    return got


def _append_plain(st):
    block, page = st["case"]["block"], st["case"]["page"]
    cu, lens, table = st["cu"].long(), st["lens"].long(), st["table"].long()
    codes, scales, x = st["codes"].view(-1, D_C), st["scales"].view(-1), st["latents"].float()
    B, per = len(lens), page // block
    t = torch.arange(len(x), device=x.device)
    seq = torch.searchsorted(cu[1:], t, right=True)
    cached = lens - (cu[1:] - cu[:-1])
    pos = cached[seq] + t - cu[seq]
    row = table[seq, pos // page] * page + pos % page
    at = row // block
    # the block that holds rows from before this call: at most the first one of each sequence
    start = cached // block * block
    old_n = cached - start
    has = (old_n > 0) & (cu[1:] > cu[:-1])
    old_row0 = table[torch.arange(B, device=x.device), start // page] * page + start % page
    old_at = old_row0 // block
    top = torch.zeros_like(scales).scatter_reduce(0, at, x.abs().amax(-1), "amax", include_self=True)
    m, e = torch.frexp(top)
    fresh = torch.ldexp(torch.ones_like(top), (e - 9 + (m > 0.875).int()).clamp(-32, 32))
    fresh = torch.where(top > 0, fresh, torch.full_like(top, 2.0 ** -32))
    was = scales[old_at]
    grown = torch.maximum(was, fresh[old_at])
    scales[at] = fresh[at]
    scales[old_at] = torch.where(has, grown, scales[old_at])
    r = torch.arange(block, device=x.device)[None, :]
    rows = torch.where((r < old_n[:, None]) & has[:, None], old_row0[:, None] + r, old_row0[:, None])
    keep = ((r < old_n[:, None]) & has[:, None])[..., None]
    held = codes[rows].float()
    held = torch.where(keep, held * torch.where(has, was / grown, torch.ones_like(was))[:, None, None], held)
    first = held[:, :1]      # rows outside the old part repeat the block's first row
    codes.view(torch.uint8)[rows] = _e4m3(torch.where(keep, held, first.expand_as(held))).view(torch.uint8)
    codes.view(torch.uint8)[row] = _e4m3(x / scales[at][:, None]).view(torch.uint8)
    return dict(codes=st["codes"], scales=st["scales"])


def _attend_plain(st):
    case = st["case"]
    page, block = case["page"], case["block"]
    n = -(-st["max_len"] // page)
    pages = st["table"][:, :n].clamp(min=0).long()
    B, H = case["batch"], case["heads"]
    c = st["codes"].view(torch.uint8)[pages].view(torch.float8_e4m3fn).float().view(B, n * page // block, block, D_C)
    c = (c * st["scales"][pages].view(B, -1, 1, 1)).view(B, n * page, D_C)
    live = torch.arange(n * page, device=c.device)[None, :] < st["lens"][:, None]
    c = torch.where(live[..., None], c, torch.zeros((), device=c.device))
    qa = torch.einsum("bhd,hdc->bhc", st["q"].float(), st["W_k"].float())
    z = torch.matmul(qa, c.transpose(1, 2)) / math.sqrt(D_H)
    z = torch.where(live[:, None, :], z, torch.full((), -math.inf, device=c.device))
    p = torch.exp(z - z.amax(-1, keepdim=True))
    lat = torch.matmul(p, c) / p.sum(-1, keepdim=True)
    o = torch.einsum("bhc,hdc->bhd", lat, st["W_v"].float())
    gate = 1 / (1 + torch.exp(-st["gate"]))
    o = o * (gate.view(B, H, D_H) if case["gate"] == "channel" else gate[..., None])
    return o.reshape(B, H * D_H).to(torch.bfloat16)


def _gated(st, dtype):
    o = st["o"].to(dtype)
    if st["gate"] is None:
        return o
    gate = 1 / (1 + torch.exp(-st["gate"].to(dtype)))
    return (o.view(len(o), gate.shape[1], -1) * gate[..., None]).reshape(o.shape)


def _w4_plain(st):
    case = st["case"]
    n, k, group = case["n"], case["heads"] * D_H, case["group"]
    code = torch.stack([st["codes"] & 15, st["codes"] >> 4], -1).view(n, k // group, group)
    w = ((code.float() - 8) * st["scales"].float()[..., None]).view(n, k)
    return torch.matmul(_gated(st, torch.float32), w.t()).to(torch.bfloat16)


# ---------------------------------------------------------------------------
# the calls that a user makes
# ---------------------------------------------------------------------------
def _model(st, **dims):
    """The layer object of a state, made once: a user's program builds it when it loads the weights."""
    if "model" not in st:
        import gated_mla_b200 as gmla
        kw = dict(d_model=1024, n_heads=16, d_h=D_H, d_c=D_C, weights={k: st[k] for k in ("W_k", "W_v") if k in st})
        st["model"] = gmla.GatedMLA(**{**kw, **dims})
        if "table" in st:
            st["cache"] = gmla.LatentCache(st["codes"], st["table"], scales=st["scales"])
        if "scales" in st and "table" not in st:
            st["w4"] = gmla.W4Weight(st["codes"], st["scales"], st["case"]["group"])
    return st["model"]


def _run_own(st):
    import gated_mla_b200 as gmla
    case = st["case"]
    op = case["op"]
    if op == "plan":
        # a serving loop keeps the plan's buffers from step to step
        p = st["plan"] = gmla.plan_batch(st["cached"], st["new"], st["table"], st["free"], st["page"], st["tokens"],
                                         out=st.get("plan"))
        return dict(block_table=st["table"], seq_lens=p.seq_lens, cu_seqlens=p.cu_seqlens, positions=p.positions,
                    seq_ids=p.seq_ids, slots=p.slots, pages_used=p.pages_used)
    if op == "norm":
        r = gmla.add_rms_norm(st["x"], st["weight"], st["residual"], eps=EPS, fp8_group=case["group"])
        got = dict(out=r.out)
        if case["residual"]:
            got["residual"] = r.residual
        if case["group"]:
            got["codes"], got["scales"] = r.codes, r.scales
        return got
    if op == "append":
        model = _model(st, cache_fp8="block")
        model.cache_append(st["latents"], st["cu"], st["lens"], st["cache"])
        return dict(codes=st["codes"], scales=st["scales"])
    if op == "attend":
        model = _model(st, n_heads=case["heads"], cache_fp8="block", gate_mode=case["gate"])
        return model.decode(st["q"], st["gate"], st["cache"], st["lens"])
    model = _model(st, d_model=case["n"], n_heads=case["heads"],
                   gate_mode=case["gate"] if case["gate"] != "none" else "channel")
    return model.gate_out_w4(st["o"], st["w4"], st["gate"])


def run(st):
    if own:
        return _run_own(st)
    op = st["case"]["op"]
    if op == "plan":
        return _plan_plain(st)
    if op == "norm":
        return _norm_plain(st)
    if op == "append":
        return _append_plain(st)
    if op == "attend":
        return _attend_plain(st)
    return _w4_plain(st)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def _mean(lo, hi):
    return (lo + hi) / 2


def work(case):
    op = case["op"]
    if op == "plan":
        b, t = case["batch"], case["batch"] * _mean(case["new_lo"], case["new_hi"]) + case["pad"]
        new_pages = case["batch"] * _mean(case["new_lo"], case["new_hi"]) / case["page"]
        return {"bytes": 8 * b + 8 * b + 16 * t + 8 * new_pages + 4 * b, "flops": 0}
    if op == "norm":
        e = 2 if case["dtype"] == "bf16" else 4
        n = case["tokens"] * case["d"]
        size = n * e * (2 + (2 if case["residual"] else 0)) + case["d"] * e
        if case["group"]:
            size += n + 4 * case["tokens"] * -(-case["d"] // case["group"])
        return {"bytes": size, "flops": 5 * n}
    if op == "append":
        t = case["batch"] * _mean(case["new_lo"], case["new_hi"])
        return {"bytes": t * D_C * 3 + 8 * case["batch"] + 4 * max(t / case["block"], case["batch"]), "flops": 2 * t * D_C}
    if op == "attend":
        lo, hi, h, b = case["len_lo"], case["len_hi"], case["heads"], case["batch"]
        tokens = b * ((hi - lo) / math.log(hi / lo) if hi > lo else hi)      # lengths are uniform in their logarithm
        gates = b * (h * D_H if case["gate"] == "channel" else h) * 4
        size = tokens * (D_C + 4 / case["block"] + 4 / case["page"]) + 2 * h * D_H * D_C * 2 + 2 * b * h * D_H * 2 + gates
        return {"bytes": size, "flops": tokens * h * D_C * 4 + 4 * b * h * D_H * D_C}
    t, n, k = case["tokens"], case["n"], case["heads"] * D_H
    gates = {"none": 0, "head": case["heads"], "channel": k}[case["gate"]] * 4 * t
    return {"bytes": n * k / 2 + 2 * n * k / case["group"] + 2 * t * (n + k) + gates, "flops": 2 * t * n * k}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _nearest_e4m3(v):
    """v rounded to the nearest value of the format: 3 fraction bits, exponents from -6, ties to even, at most 448."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -60)))
    e = torch.where(torch.ldexp(torch.ones_like(v), e.int()) > v.abs(), e - 1, e)      # log2 next to a power of two
    e = torch.where(torch.ldexp(torch.ones_like(v), e.int() + 1) <= v.abs(), e + 1, e)
    step = torch.ldexp(torch.ones_like(v), (e.clamp(min=-6) - 3).int())
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "plan":
        return None        # whole numbers only
    if op == "norm":
        s = st["x"].double() + (st["residual"].double() if case["residual"] else 0)
        y = st["weight"].double() * s / torch.sqrt((s * s).sum(1, keepdim=True) / case["d"] + EPS)
        got = dict(out=y)
        if case["residual"]:
            got["residual"] = s
        if case["group"]:
            parts = [y[:, i:i + case["group"]] for i in range(0, case["d"], case["group"])]
            got["scales"] = torch.stack([q.abs().amax(1) for q in parts], 1) / E4M3_MAX
            got["scales"] = torch.where(got["scales"] > 0, got["scales"], torch.ones_like(got["scales"]))
            got["codes"] = torch.cat([_nearest_e4m3(q / got["scales"][:, i:i + 1]) for i, q in enumerate(parts)], 1)
        return got
    if op == "append":
        codes, scales = st["codes"].double().view(-1, D_C), st["scales"].double().view(-1)
        cu, lens, table, block, page = st["cu"].tolist(), st["lens"].tolist(), st["table"].tolist(), case["block"], case["page"]
        x = st["latents"].double()
        for b, n in enumerate(lens):
            pos = n - (cu[b + 1] - cu[b])
            while pos < n:
                upto = min(n, pos // block * block + block)
                lo = table[b][pos // page] * page + pos // block * block % page
                held, new = pos % block, x[cu[b + 1] - (n - pos):cu[b + 1] - (n - upto)]
                top, scale = float(new.abs().max()), 2.0 ** -32
                while top > E4M3_MAX * scale and scale < 2.0 ** 32:
                    scale *= 2
                if held:
                    was = float(scales[lo // block])
                    scale = max(scale, was)
                    codes[lo:lo + held] = _nearest_e4m3(codes[lo:lo + held] * (was / scale))
                codes[lo + held:lo + held + len(new)] = _nearest_e4m3(new / scale)
                scales[lo // block] = scale
                pos = upto
        return dict(codes=codes.view(st["codes"].shape), scales=scales.view(st["scales"].shape))
    if op == "attend":
        H, page, rows = case["heads"], case["page"], []
        for b, n in enumerate(st["lens"].tolist()):
            ids = st["table"][b, :-(-n // page)].long()
            c = st["codes"].view(torch.uint8)[ids].view(torch.float8_e4m3fn).double().view(-1, case["block"], D_C)
            c = (c * st["scales"][ids].double().view(-1, 1, 1)).view(-1, D_C)[:n]
            k = torch.matmul(st["q"][b].double()[:, None, :], st["W_k"].double())[:, 0]
            a = torch.softmax(torch.matmul(c, k.t()).t() / math.sqrt(D_H), -1)
            rows.append(torch.matmul(st["W_v"].double(), torch.matmul(a, c)[..., None])[..., 0])
        o = torch.stack(rows)
        gate = torch.sigmoid(st["gate"].double())
        return (o * (gate.view(o.shape) if case["gate"] == "channel" else gate[..., None])).reshape(len(rows), H * D_H)
    code = torch.empty(case["n"], case["heads"] * D_H, dtype=torch.float64, device="cuda")
    code[:, 0::2], code[:, 1::2] = (st["codes"] % 16).double() - 8, (st["codes"] // 16).double() - 8
    w = code * st["scales"].double().repeat_interleave(case["group"], 1)
    return _gated(st, torch.float64) @ w.t()
