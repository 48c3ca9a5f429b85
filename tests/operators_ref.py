"""Plain 64-bit forms of the operators around a decode step (test helper): sequential,
on the CPU, written from the formulas in include/gmla.h. No code is shared with
the library."""
from __future__ import annotations

import numpy as np
import torch

E4M3_MAX = 448.0


def e4m3(v: np.ndarray) -> np.ndarray:
    """Nearest E4M3 values (ties to even, saturating), as float64."""
    v = np.asarray(v, dtype=np.float64)
    a = np.abs(v)
    e = np.floor(np.log2(np.maximum(a, 2.0 ** -60)))
    e = np.where(2.0 ** e > a, e - 1, e)
    e = np.where(2.0 ** (e + 1) <= a, e + 1, e)
    step = 2.0 ** (np.maximum(e, -6) - 3)
    return np.clip(np.round(v / step) * step, -E4M3_MAX, E4M3_MAX)


def e4m3_codes(v: np.ndarray) -> np.ndarray:
    """Codes (uint8) of values that lie on the E4M3 grid."""
    return torch.from_numpy(np.ascontiguousarray(v, np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def e4m3_values(codes: np.ndarray) -> np.ndarray:
    return torch.from_numpy(np.ascontiguousarray(codes)).view(torch.float8_e4m3fn).to(torch.float32).numpy().astype(np.float64)


def plan(cached, new, table, free, page, T):
    """The step plan, request by request. Returns a dict of int arrays; `table` is not changed."""
    table = np.array(table)
    B = len(cached)
    pos = np.full(T, -1, np.int32)
    seq = np.full(T, -1, np.int32)
    slot = np.full(T, -1, np.int64)
    cu = np.zeros(B + 1, np.int32)
    used = t = 0
    for b in range(B):
        for i in range(new[b]):
            p = cached[b] + i
            if p % page == 0:
                table[b, p // page] = free[used]
                used += 1
            pos[t], seq[t], slot[t] = p, b, int(table[b, p // page]) * page + p % page
            t += 1
        cu[b + 1] = t
    return dict(table=table, seq_lens=np.asarray(cached) + np.asarray(new), cu_seqlens=cu, positions=pos, seq_ids=seq,
                slots=slot, pages_used=used)


def block_scale(top: float) -> float:
    """2^E with the smallest E in [-32, 32] for which top <= 448 * 2^E."""
    s = 2.0 ** -32
    while top > E4M3_MAX * s and s < 2.0 ** 32:
        s *= 2
    return s


def append(codes, scales, row_of, block_of, latents, cu, lens, block):
    """Append in place: codes [rows, 512] float64 values, scales float64 [blocks]."""
    for b in range(len(lens)):
        p = lens[b] - (cu[b + 1] - cu[b])
        t = cu[b]
        while p < lens[b]:
            end = min(lens[b], p // block * block + block)
            new = latents[t:t + end - p]
            s = block_scale(np.abs(new).max())
            at = block_of(b, p)
            if p % block:
                first = row_of(b, p // block * block)
                s = max(s, scales[at])
                held = slice(first, first + p % block)
                codes[held] = e4m3(codes[held] * (scales[at] / s))
            r = row_of(b, p)
            codes[r:r + end - p] = e4m3(new / s)
            scales[at] = s
            t += end - p
            p = end


def gate_values(logits, mode, H, d_h, topk=0):
    """Gate of every output channel [B, H * d_h] in 64 bits."""
    z = np.asarray(logits, np.float64)
    if mode == "channel":
        return 1 / (1 + np.exp(-z))
    if mode == "head":
        g = 1 / (1 + np.exp(-z))
    elif mode == "head_topk":
        g = np.zeros_like(z)
        for b in range(len(z)):
            g[b, np.argsort(-z[b], kind="stable")[:topk]] = 1
    elif mode == "head_binary":
        g = (z >= 0).astype(np.float64)
    else:
        g = np.where(z < -np.log(3.0), 0.0, np.where(z < np.log(3.0), 0.5, 1.0))
    return np.repeat(g, d_h, axis=1)


def decode(q, c, W_k, W_v, scale, s):
    """One query [H, d_h] over rows c [L, d_c] whose codes have scales s [L]. Returns (o [H, d_h], bound [H, d_h]).

    The bound covers the roundings of an FP8 decode, to first order in each:
      * the absorbed query is a sum of two E4M3 terms: relative 2^-4 * 2^-4 an element (and
        2^-19 of the largest, the second term's subnormal step), so a score is off by at
        most d = scale * (2^-8 sum |q_i c_i| + 2^-19 max|q| sum |c_i|), and a weight by a
        factor within e^(2 d) of 1;
      * three E4M3 terms, each 32 times finer, hold a weight times its row's scale to 2^-12 (half a
        step three times: 2^-4 * 2^-4 * 2^-4), and to half the last subnormal step below that:
        2^-10 / 32^2 of 8 times the reference, which is at most the largest: 2^-23 of it;
      * the latent sum is rounded to bf16 (half a step, 2^-8), and so is the result;
      * fp32 sums of up to L terms, and the hardware exponential and logarithm: 2^-18.
    """
    H = q.shape[0]
    o = np.zeros((H, W_v.shape[1]))
    bound = np.zeros_like(o)
    if not len(c):
        return o, bound
    ac = np.abs(c)
    for h in range(H):
        qa = q[h] @ W_k[h]
        z = c @ qa * scale
        dz = scale * (2.0 ** -8 * (ac @ np.abs(qa)) + 2.0 ** -19 * np.abs(qa).max() * ac.sum(1))
        p = np.exp(z - z.max())
        p /= p.sum()
        lat = p @ c
        mag = p @ ac                                     # sum p |c|
        wd = (p * np.expm1(np.minimum(2 * dz, 50))) @ ac + np.abs(lat) * (p @ np.expm1(np.minimum(2 * dz, 50)))
        d_lat = wd + mag * (2.0 ** -12 + 2.0 ** -18) + 2.0 ** -23 * (p * s).max() * (ac / s[:, None]).sum(0) + 2.0 ** -8 * np.abs(lat)
        o[h] = W_v[h] @ lat
        bound[h] = np.abs(W_v[h]) @ d_lat + 2.0 ** -8 * np.abs(o[h]) + 2.0 ** -18 * (np.abs(W_v[h]) @ np.abs(lat))
    return o, bound


def w4_dense(codes, scales, group):
    """[N, K] in 64 bits."""
    N, half = codes.shape
    w = np.empty((N, 2 * half))
    w[:, 0::2] = (codes & 15).astype(np.float64) - 8
    w[:, 1::2] = (codes >> 4).astype(np.float64) - 8
    return w * np.repeat(np.asarray(scales, np.float64), group, axis=1)
