"""The operators around a decode step reject bad arguments before any device work (no GPU needed)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def L():
    from gated_mla_b200 import _lib
    return _lib


P = 0x10000     # an aligned address that no accepted call gets to use


def _cfg(L, **kw):
    c = L.gmla_config()
    c.d_model, c.n_heads, c.d_h, c.d_c, c.d_rope = 2048, 16, 128, 512, 0
    c.gate_mode, c.gate_bias, c.softmax_scale, c.rope_base, c.dtype = 0, 0, 128 ** -0.5, 1e4, 0
    c.cache_dtype = L.GMLA_CACHE_FP8_BLOCK
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _cache(L, **kw):
    k = L.gmla_cache()
    k.data, k.batch, k.capacity, k.scales, k.scale_block = P, 4, 256, P, 64
    for n, v in kw.items():
        setattr(k, n, v)
    return k


def _plan(L, **kw):
    a = dict(cached_lens=P, new_lens=P + 256, B=2, free_pages=P, n_free=4, page_size=16, block_table=P, max_pages_per_seq=4, T=8,
             seq_lens=P + 512, cu_seqlens=P + 768, positions=P, seq_ids=P, slots=P, pages_used=P, ws=P, ws_bytes=256, stream=None)
    a.update(kw)
    return L.gmla_plan_batch(*a.values())


@pytest.mark.parametrize("bad", [dict(B=-1), dict(T=-1), dict(n_free=-1), dict(page_size=0), dict(max_pages_per_seq=0),
                                 dict(cached_lens=None), dict(new_lens=None), dict(free_pages=None), dict(block_table=None),
                                 dict(seq_lens=None), dict(cu_seqlens=None), dict(positions=P + 4), dict(slots=P + 8),
                                 dict(seq_ids=None), dict(pages_used=None), dict(cached_lens=P + 1), dict(new_lens=P + 2),
                                 dict(free_pages=P + 2), dict(seq_lens=P), dict(seq_lens=P + 256), dict(cu_seqlens=P),
                                 dict(cu_seqlens=P + 256), dict(cached_lens=P + 516), dict(new_lens=P + 776)])
def test_plan_batch(L, bad):
    assert _plan(L, **bad) == L.GMLA_ERR_INVALID_ARG


def test_plan_batch_workspace_and_range(L):
    assert _plan(L, ws=None) == L.GMLA_ERR_WORKSPACE
    assert _plan(L, ws_bytes=255) == L.GMLA_ERR_WORKSPACE
    assert _plan(L, page_size=1 << 20, max_pages_per_seq=1 << 12) == L.GMLA_ERR_UNSUPPORTED
    assert _plan(L, T=(1 << 30) + 1) == L.GMLA_ERR_UNSUPPORTED


def _norm(L, **kw):
    a = dict(dtype=0, x=P, x_stride=64, residual=P, residual_stride=64, weight=P, eps=1e-6, T=4, d=64, residual_out=P + 4096,
             residual_out_stride=64, out=P, out_stride=64, codes=P, scales=P, group=32, stream=None)
    a.update(kw)
    return L.gmla_add_rms_norm(*a.values())


@pytest.mark.parametrize("bad", [dict(dtype=2), dict(T=-1), dict(d=0), dict(eps=-1.0), dict(eps=float("inf")), dict(group=16),
                                 dict(group=-32), dict(group=0), dict(codes=None), dict(scales=None), dict(x=None),
                                 dict(x=P + 2), dict(residual_out=P), dict(x_stride=63), dict(out_stride=0), dict(residual_stride=-64),
                                 dict(out=None, residual_out=None, codes=None, scales=None, group=0)])
def test_add_rms_norm(L, bad):
    assert _norm(L, **bad) == L.GMLA_ERR_INVALID_ARG


def test_add_rms_norm_width(L):
    assert _norm(L, d=32769, x_stride=40000) == L.GMLA_ERR_UNSUPPORTED
    assert _norm(L, T=0) == L.GMLA_OK


def _append(L, cfg=None, cache=None, **kw):
    a = dict(latents=P, stride=512, cu=P, lens=P, B=2, T=4, ws=P, ws_bytes=256, s=None)
    a.update(kw)
    return L.gmla_cache_append(cfg or _cfg(L), cache or _cache(L), *a.values())


@pytest.mark.parametrize("bad", [dict(B=-1), dict(T=-1), dict(latents=None), dict(latents=P + 8), dict(cu=None), dict(lens=None),
                                 dict(stride=511), dict(stride=516), dict(B=5)])
def test_cache_append(L, bad):
    assert _append(L, **bad) == L.GMLA_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(scales=None), dict(scales=P + 4), dict(scale_block=0), dict(scale_block=48),
                                 dict(scale_block=256), dict(scale_block=-1), dict(data=None),
                                 dict(paged=1, block_table=P, page_size=32, num_pages=4, max_pages_per_seq=4)])
def test_block_scaled_cache(L, bad):
    k = _cache(L, **bad)
    assert _append(L, cache=k) == L.GMLA_ERR_INVALID_ARG
    w = L.gmla_weights()
    assert L.gmla_decode(_cfg(L), w, P, None, k, P, 2, P, P, 1 << 30, None) == L.GMLA_ERR_INVALID_ARG


def test_block_scaled_cache_where_it_is_not_covered(L):
    w = L.gmla_weights()
    assert _append(L, cfg=_cfg(L, cache_dtype=L.GMLA_CACHE_SAME)) == L.GMLA_ERR_UNSUPPORTED
    assert _append(L, cfg=_cfg(L, d_rope=64)) == L.GMLA_ERR_UNSUPPORTED
    assert _append(L, cfg=_cfg(L, d_c=256)) == L.GMLA_ERR_UNSUPPORTED
    assert _append(L, cfg=_cfg(L, dtype=1)) == L.GMLA_ERR_INVALID_ARG
    assert _append(L, cfg=_cfg(L, cache_dtype=3)) == L.GMLA_ERR_INVALID_ARG
    assert _append(L, ws=None) == L.GMLA_ERR_WORKSPACE
    assert L.gmla_latent_project(_cfg(L), w, P, 4, P, P, _cache(L), P, P, P, 1 << 20, None) == L.GMLA_ERR_UNSUPPORTED
    assert L.gmla_prefill(_cfg(L), w, P, None, _cache(L), P, 1, 4, 4, P, P, 1 << 30, None) == L.GMLA_ERR_UNSUPPORTED
    for bad in (dict(n_heads=0), dict(dtype=1)):
        assert L.gmla_decode_workspace_size(_cfg(L, **bad), 4) == 256


def _w4(L, cfg=None, group=64, codes=P, scales=P, **kw):
    s = L.gmla_w4()
    s.codes, s.scales, s.group = codes, scales, group
    a = dict(o=P, T=2, gate=None, y=P, ws=P, ws_bytes=1 << 30, stream=None)
    a.update(kw)
    return L.gmla_gate_out_w4(cfg or _cfg(L, cache_dtype=0), s, *a.values())


@pytest.mark.parametrize("bad", [dict(group=0), dict(group=48), dict(group=256), dict(T=-1), dict(o=None), dict(y=P + 2),
                                 dict(codes=None), dict(scales=P + 2), dict(gate=P + 4)])
def test_gate_out_w4(L, bad):
    assert _w4(L, **bad) == L.GMLA_ERR_INVALID_ARG


def test_gate_out_w4_sizes(L):
    assert _w4(L, cfg=_cfg(L, cache_dtype=0, n_heads=1, d_h=64), group=128) == L.GMLA_ERR_INVALID_ARG
    assert _w4(L, cfg=_cfg(L, cache_dtype=0, dtype=1)) == L.GMLA_ERR_UNSUPPORTED
    assert _w4(L, cfg=_cfg(L, cache_dtype=0, d_h=12, n_heads=16)) == L.GMLA_ERR_UNSUPPORTED
    assert _w4(L, ws_bytes=256) == L.GMLA_ERR_WORKSPACE
    assert _w4(L, T=0) == L.GMLA_OK
    c = _cfg(L, cache_dtype=0)
    assert L.gmla_gate_out_w4_workspace_size(c, 1) >= 256 + 2 * 2048
    assert L.gmla_gate_out_w4_workspace_size(c, 65) >= 256 + 65 * 2 * 2048
    assert L.gmla_gate_out_w4_workspace_size(_cfg(L, d_h=0), 1) == 256
    assert L.gmla_gate_out_w4_workspace_size(c, -1) == 256


def test_null_structures(L):
    w4 = L.gmla_w4()
    f = L.lib.gmla_gate_out_w4
    assert f(None, ctypes.byref(w4), P, 1, None, P, P, 1 << 20, None) == L.GMLA_ERR_INVALID_ARG
    c = _cfg(L, cache_dtype=0)
    assert f(ctypes.byref(c), None, P, 1, None, P, P, 1 << 20, None) == L.GMLA_ERR_INVALID_ARG
    assert L.lib.gmla_cache_append(ctypes.byref(_cfg(L)), None, P, 512, P, P, 1, 1, P, 256, None) == L.GMLA_ERR_INVALID_ARG


def test_python_checks_without_a_gpu():
    import torch

    import gated_mla_b200 as gmla
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        gmla.add_rms_norm(x)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        gmla.plan_batch(i, i, i.view(4, 1), i, 16, 4)
    with pytest.raises(ValueError):
        gmla.quantize_w4(torch.zeros(4, 100), 64)
    with pytest.raises(ValueError):
        gmla.GatedMLA(d_model=64, n_heads=1, d_h=128, d_c=512, weights={}, cache_fp8="rows")
