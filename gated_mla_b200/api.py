"""Torch-facing marshalling over the C ABI (device memory and streams only).

``GatedMLA`` holds a configuration and device weight tensors and exposes the
library's calls on a layer. ``plan_batch`` (block table, positions and slots of a
step) and ``add_rms_norm`` stand beside it, and ``W4Weight`` / ``quantize_w4`` hold a
weight in 4 bits. Outputs and workspaces are torch allocations; every
computation happens inside libgmla.so on the current CUDA stream.
"""
from __future__ import annotations

import dataclasses
import math
import threading
import weakref
from typing import NamedTuple, Optional

import torch

from . import _lib as L

_DT = {torch.bfloat16: L.GMLA_BF16, torch.float32: L.GMLA_FP32}
_GATE = {"channel": L.GMLA_GATE_CHANNEL, "head": L.GMLA_GATE_HEAD, "head_topk": L.GMLA_GATE_HEAD_TOPK,
         "head_binary": L.GMLA_GATE_HEAD_BINARY, "head_ternary": L.GMLA_GATE_HEAD_TERNARY}


def _p(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("gated_mla_b200 takes CUDA tensors only")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


@dataclasses.dataclass
class LatentCache:
    """Latent cache rows [c | k^R] (contiguous [B, cap, row] or paged [pages, page, row])."""
    data: torch.Tensor
    block_table: Optional[torch.Tensor] = None   # int32 [B, max_pages_per_seq] for paged
    batch: int = 0
    # block-scaled FP8 cache: fp32, one scale for each block of scale_block rows
    # ([pages, page // block] for paged, [B, ceil(cap / block)] for contiguous)
    scales: Optional[torch.Tensor] = None
    scale_block: int = 0          # 0 with a paged cache: page // scales.shape[1]

    @property
    def paged(self) -> bool:
        return self.block_table is not None

    def struct(self) -> L.gmla_cache:
        data, table, scales = self.data, self.block_table, self.scales
        shape = data.shape
        n, rows = shape[0], shape[1]
        block = self.scale_block
        if scales is not None:
            if not block:
                if table is None:
                    raise ValueError("a contiguous block-scaled cache needs scale_block")
                block = rows // max(scales.shape[1], 1)
            if (scales.dtype is not torch.float32 or scales.device != data.device or block < 1
                    or scales.shape != (n, -(-rows // block))):
                raise ValueError("scales must be float32 [pages, page // block] (paged) or [B, ceil(capacity / block)] "
                                 "on the cache's device")
        else:
            block = 0
        if table is None:
            return L.gmla_cache(_p(data), 0, n, rows, 0, 0, 0, None, _p(scales), block)
        B, M = table.shape
        return L.gmla_cache(_p(data), 1, B, M * rows, rows, n, M, _p(table), _p(scales), block)


def _check(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple, device: torch.device) -> None:
    """A tensor argument of the calls below: its type, its sizes and its device."""
    if t.dtype is not dtype or t.shape != shape or t.device != device:
        raise ValueError(f"{name} must be {dtype} {list(shape)} on {device}, got {t.dtype} {list(t.shape)} on {t.device}")


# the current stream's handle without a Stream object around it (3 us less a call)
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice     # of a process whose CUDA context exists: a CUDA tensor is at hand


def _stream_of(t: torch.Tensor) -> int:
    """The current stream, which has to be one of the tensor's device."""
    if not t.is_cuda:
        raise ValueError("gated_mla_b200 takes CUDA tensors only")
    index = t.get_device()
    if index != _current_device():
        raise ValueError(f"the tensors are on {t.device}, the current device is cuda:{torch.cuda.current_device()}: "
                         "call inside torch.cuda.device(...)")
    return _raw_stream(index)


class _Memory:
    """256 bytes of the library's device memory, for torch."""

    def __init__(self, address: int):
        self.__cuda_array_interface__ = dict(shape=(256,), typestr="|u1", data=(address, False), version=3)


class _Scratch:
    """Device memory of the calls. Workspaces go by (call, device, stream): calls on different
    streams never share one, and a call under graph capture gets one of its own, which belongs to
    that graph. Status words go by (call, device) and stay: captured calls record their faults in
    them too, where sync_status finds them.

    `lock` is held from get() to the end of the call that uses the workspace: threads that share a
    stream then share its workspaces too, one call's kernels enqueued whole before the next's."""

    def __init__(self):
        self._held = {}
        self.lock = threading.Lock()

    def get(self, key: str, nbytes: int, device: torch.device, stream: int) -> torch.Tensor:
        """At least `nbytes` bytes, of any content."""
        if torch.cuda.is_current_stream_capturing():
            return torch.empty(nbytes, dtype=torch.uint8, device=device)
        ws = self._held.get((key, device.index, stream))
        if ws is None or ws.numel() < nbytes:
            ws = self._held[(key, device.index, stream)] = torch.empty(nbytes, dtype=torch.uint8, device=device)
        return ws

    def word(self, key: str, device: torch.device) -> torch.Tensor:
        """256 bytes that begin with a status word, zero at first."""
        word = self._held.get((key, device.index))
        if word is None:
            with self.lock, torch.cuda.device(device):
                word = self._held.get((key, device.index))      # another thread's, by now
                if word is None:
                    word = self._held[(key, device.index)] = torch.as_tensor(_Memory(L.gmla_status_word()), device=device)
        return word

    def words(self):
        return [(key[0], ws) for key, ws in list(self._held.items()) if len(key) == 2]

    def sync_status(self) -> None:
        for key, word in self.words():
            with torch.cuda.device(word.device):
                torch.cuda.synchronize()
                L.check(L.gmla_sync_status(word.data_ptr(), None), f"device status ({key})")

    def clear_status(self) -> None:
        for _, word in self.words():
            with torch.cuda.device(word.device):
                torch.cuda.synchronize()       # what was launched before is not to report afterwards
                L.check(L.gmla_clear_status(word.data_ptr(), None), "clear_status")
                torch.cuda.synchronize()


_scratch = _Scratch()
_layers_scratch = lambda: None       # noqa: E731  (a weak reference once there is a layer)


def _shared_scratch() -> _Scratch:
    """The workspaces that all layers share, as long as there are any: the largest workspace of a call
    holds a whole weight (gate_out_w4 above 256 tokens), which a model has room for once, not in each layer."""
    global _layers_scratch
    shared = _layers_scratch()
    if shared is None:
        shared = _Scratch()
        _layers_scratch = weakref.ref(shared)
    return shared


def sync_status() -> None:
    """Synchronise and raise if a plan_batch call, captured ones included, reported a batch that cannot
    be. The report stays until clear_status."""
    _scratch.sync_status()


def clear_status() -> None:
    """Synchronise and forget what plan_batch calls have reported."""
    _scratch.clear_status()


class BatchPlan:
    """What one step of a batch over a paged cache needs (see plan_batch)."""
    __slots__ = ("seq_lens", "cu_seqlens", "positions", "seq_ids", "slots", "pages_used", "_sizes")

    def __init__(self, batch: int, n_tokens: int, device: torch.device):
        def new(n, dtype=torch.int32):
            return torch.empty(n, dtype=dtype, device=device)
        self.seq_lens = new(batch)                      # int32 [B]: rows of each sequence, the new ones included
        self.cu_seqlens = new(batch + 1)                # int32 [B + 1]: packed token offsets
        self.positions = new(n_tokens)                  # int32 [n_tokens], -1 behind the last sequence
        self.seq_ids = new(n_tokens)                    # int32 [n_tokens]
        self.slots = new(n_tokens, torch.int64)         # int64 [n_tokens]: page * page_size + row
        self.pages_used = new(1)                        # int32 [1]: how many of the free pages were taken
        self._sizes = (batch, n_tokens, device)


def plan_batch(cached_lens: torch.Tensor, new_lens: torch.Tensor, block_table: torch.Tensor, free_pages: torch.Tensor,
               page_size: int, n_tokens: int, out: Optional[BatchPlan] = None) -> BatchPlan:
    """The plan of one step, made on the GPU from its request lengths.

    ``cached_lens`` and ``new_lens`` are int32 [B]; ``block_table`` (int32 [B, max_pages])
    gets the entries of the pages that new rows begin, taken from ``free_pages`` in the
    order of the sequences. ``n_tokens`` is the number of token rows, at least the sum of
    new_lens; rows behind the last sequence get -1. ``out`` reuses the buffers of an
    earlier plan of the same sizes (copy its ``seq_lens`` first when they are this
    step's ``cached_lens``). A batch that does not fit is planned as empty and
    reported by ``sync_status`` until ``clear_status``.
    """
    dev, B, T = cached_lens.device, cached_lens.shape[0], n_tokens
    stream = _stream_of(cached_lens)
    if block_table.dim() != 2 or free_pages.dim() != 1 or T < 0:
        raise ValueError("block_table is [B, max_pages], free_pages [n], n_tokens >= 0")
    M, n_free = block_table.shape[1], free_pages.shape[0]
    i32 = torch.int32
    _check(cached_lens, "cached_lens", i32, (B,), dev)
    _check(new_lens, "new_lens", i32, (B,), dev)
    _check(block_table, "block_table", i32, (B, M), dev)
    _check(free_pages, "free_pages", i32, (n_free,), dev)
    if out is None:
        out = BatchPlan(B, T, dev)
    elif out._sizes != (B, T, dev):
        raise ValueError(f"out is a plan of {out._sizes}, this batch is {(B, T, dev)}")
    ws = _scratch.word("plan_batch", dev)
    L.check(L.lib.gmla_plan_batch(
        _p(cached_lens), _p(new_lens), B, _p(free_pages), n_free, page_size, _p(block_table), M, T,
        out.seq_lens.data_ptr(), out.cu_seqlens.data_ptr(), out.positions.data_ptr(), out.seq_ids.data_ptr(),
        out.slots.data_ptr(), out.pages_used.data_ptr(), ws.data_ptr(), 256, stream), "gmla_plan_batch")
    return out


class NormOut(NamedTuple):
    """Outputs of add_rms_norm; those not asked for are None."""
    out: Optional[torch.Tensor]        # [T, d]: the normalised rows
    residual: Optional[torch.Tensor]   # [T, d]: x + residual
    codes: Optional[torch.Tensor]      # float8_e4m3fn [T, d]
    scales: Optional[torch.Tensor]     # float32 [T, ceil(d / group)]


def add_rms_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None, *,
                 eps: float = 1e-6, fp8_group: int = 0, out: Optional[torch.Tensor] = None,
                 residual_out: Optional[torch.Tensor] = None, want_out: bool = True) -> NormOut:
    """s = x + residual, y = s / sqrt(mean(s^2) + eps) * weight, over the rows of x [T, d].

    Rows may be strided (their elements contiguous). With ``fp8_group`` (32, 64, 128 or
    256) y also comes as E4M3 codes with one scale for each group of columns;
    ``want_out=False`` then leaves the unquantised y out. ``residual_out`` and ``out`` may be
    ``residual`` or ``x`` itself (one each); any other overlap is refused.
    """
    stream = _stream_of(x)
    if x.dtype not in _DT or x.dim() != 2:
        raise ValueError("x must be bfloat16 or float32 [T, d]")
    dev, (T, d) = x.device, x.shape
    if residual is None and residual_out is not None:
        raise ValueError("residual_out goes with a residual")

    def row(t, name):      # address and row stride
        if t is None:
            return None, 0
        if t is not x:
            _check(t, name, x.dtype, (T, d), dev)
        if t.is_contiguous():
            return t.data_ptr(), d
        if d > 1 and t.stride(1) != 1:
            raise ValueError(f"{name}: the elements of a row must be contiguous")
        return t.data_ptr(), t.stride(0) if T > 1 else d

    if out is None and want_out:
        out = x.new_empty((T, d))
        out_row = out.data_ptr(), d
    else:
        out_row = row(out, "out")
    if residual is not None and residual_out is None:
        residual_out = x.new_empty((T, d))
        sum_row = residual_out.data_ptr(), d
    else:
        sum_row = row(residual_out, "residual_out")
    codes = scales = codes_at = scales_at = None
    if fp8_group:
        if fp8_group < 0:
            raise ValueError("fp8_group must be 0, 32, 64, 128 or 256")
        codes = x.new_empty((T, d), dtype=torch.float8_e4m3fn)
        scales = x.new_empty((T, -(-d // fp8_group)), dtype=torch.float32)
        codes_at, scales_at = codes.data_ptr(), scales.data_ptr()
    if weight is not None:
        _check(weight, "weight", x.dtype, (d,), dev)
    L.check(L.lib.gmla_add_rms_norm(_DT[x.dtype], *row(x, "x"), *row(residual, "residual"), _p(weight), eps, T, d,
                                *sum_row, *out_row, codes_at, scales_at, fp8_group, stream), "gmla_add_rms_norm")
    return NormOut(out, residual_out, codes, scales)


@dataclasses.dataclass
class W4Weight:
    """A weight matrix [N, K] in 4 bits: W[n, k] = (code - 8) * scales[n, k // group]."""
    codes: torch.Tensor       # uint8 [N, K // 2], even k in the low nibble
    scales: torch.Tensor      # bfloat16 [N, K // group]
    group: int = 128

    def struct(self) -> L.gmla_w4:
        w = L.gmla_w4()
        w.codes, w.scales, w.group = _p(self.codes), _p(self.scales), self.group
        return w


def quantize_w4(weight: torch.Tensor, group: int = 128) -> W4Weight:
    """Nearest 4-bit codes of a weight [N, K], the scale of a group its largest magnitude / 7 (done once, at load time)."""
    N, K = weight.shape
    if group not in (32, 64, 128) or K % group:
        raise ValueError("group must be 32, 64 or 128 and divide K")
    w = weight.float().view(N, K // group, group)
    scales = (w.abs().amax(-1) / 7).to(torch.bfloat16)
    step = scales.float().unsqueeze(-1)
    code = torch.where(step > 0, torch.round(w / step), torch.zeros((), device=w.device)).clamp(-8, 7) + 8
    code = code.to(torch.uint8).view(N, K)
    return W4Weight((code[:, 0::2] | (code[:, 1::2] << 4)).contiguous(), scales.contiguous(), group)


class GatedMLA:
    def __init__(self, *, d_model: int, n_heads: int, d_h: int, d_c: int, d_rope: int = 0,
                 gate_mode: str = "channel", softmax_scale: Optional[float] = None,
                 rope_base: float = 10000.0, dtype: torch.dtype = torch.bfloat16,
                 weights: dict, d_cq: int = 0, gate_topk: int = 0, cache_fp8=False,
                 cache_scale: float = 1.0):
        # cache_fp8: False, True (E4M3 codes, one scale for the cache) or "block" (one scale for each block of rows)
        if cache_fp8 not in (False, True, "block"):
            raise ValueError("cache_fp8 must be False, True or 'block'")
        self.dtype = dtype
        self.cfg = L.gmla_config()
        self.cfg.d_model, self.cfg.n_heads, self.cfg.d_h, self.cfg.d_c, self.cfg.d_rope = (
            d_model, n_heads, d_h, d_c, d_rope)
        self.cfg.gate_mode = _GATE[gate_mode]
        self.cfg.gate_topk = gate_topk
        self.cfg.gate_bias = 1 if weights.get("b_g") is not None else 0
        self.cfg.softmax_scale = softmax_scale if softmax_scale else 1.0 / math.sqrt(d_h + d_rope)
        self.cfg.rope_base = rope_base
        self.cfg.dtype = _DT[dtype]
        self.cfg.d_cq = d_cq
        self.cfg.cache_dtype = (L.GMLA_CACHE_FP8_BLOCK if cache_fp8 == "block"
                                else L.GMLA_CACHE_FP8_E4M3 if cache_fp8 else L.GMLA_CACHE_SAME)
        self.cfg.cache_scale = cache_scale
        self.weights = dict(weights)
        self.w = L.gmla_weights()
        for k in ("W_c", "W_kr", "W_q", "W_qr", "W_k", "W_v", "W_g", "b_g", "W_o", "W_dq", "W_uq"):
            setattr(self.w, k, _p(self.weights.get(k)))
        self._ws = {}
        self._scratch = _shared_scratch()     # workspaces of the calls that report into the layer's word
        self._status = _Scratch()             # that word
        self._status_on = -1                  # the device whose word the configuration names
        self._staging_cfg = None

    # -- sizes
    @property
    def G(self) -> int:
        return self.cfg.n_heads * self.cfg.d_h if self.cfg.gate_mode == L.GMLA_GATE_CHANNEL else self.cfg.n_heads

    @property
    def row(self) -> int:
        return self.cfg.d_c + self.cfg.d_rope

    def workspace(self, key: str, nbytes: int, device) -> torch.Tensor:
        ws = self._ws.get(key)
        if ws is None or ws.numel() < nbytes:
            ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
            self._ws[key] = ws
            L.check(L.gmla_clear_status(ws.data_ptr(), torch.cuda.current_stream().cuda_stream), "clear_status")
        return ws

    def _status_cfg(self, device: torch.device, staging: bool = False) -> L.gmla_config:
        """The configuration with the layer's status word on the device; `staging`: the same layer over a bf16 cache."""
        if self._status_on != device.index:
            self.cfg.status = self._status.word("layer", device).data_ptr()
            self._status_on, self._staging_cfg = device.index, None
        if not staging:
            return self.cfg
        if self._staging_cfg is None:
            cfg = L.gmla_config.from_buffer_copy(self.cfg)
            cfg.cache_dtype = L.GMLA_CACHE_SAME
            self._staging_cfg = cfg
        return self._staging_cfg

    @staticmethod
    def _stream() -> int:
        return _raw_stream(torch.cuda.current_device())

    # -- the four calls
    @property
    def block_scaled(self) -> bool:
        return self.cfg.cache_dtype == L.GMLA_CACHE_FP8_BLOCK

    def latent_project(self, x, positions, seq_ids, cache: LatentCache, q_out=None, gate_logits=None, *,
                       cu_seqlens=None, seq_lens=None):
        """Project the tokens and write their latents into the cache; nothing is cached for padding
        (tokens with position and seq_id -1, as plan_batch marks them). A block-scaled cache
        takes the packing of the tokens too (``cu_seqlens`` and ``seq_lens``, as cache_append):
        the latents go through a bf16 buffer of the step's rows."""
        T = x.shape[0]
        c = self.cfg
        if self.block_scaled:
            return self._project_and_append(x, cache, q_out, gate_logits, cu_seqlens, seq_lens)
        if q_out is None:
            q_out = torch.empty(T, c.n_heads, c.d_h + c.d_rope, dtype=self.dtype, device=x.device)
        if gate_logits is None:
            gate_logits = torch.empty(T, self.G, dtype=torch.float32, device=x.device)
        nb = L.gmla_latent_project_workspace_size(c, T)
        ws = self.workspace("project", nb, x.device)
        L.check(L.gmla_latent_project(c, self.w, _p(x), T, _p(positions), _p(seq_ids), cache.struct(),
                                      _p(q_out), _p(gate_logits), ws.data_ptr(), ws.numel(), self._stream()),
                "gmla_latent_project")
        return q_out, gate_logits

    def decode(self, q, gate_logits, cache: LatentCache, seq_lens, o_out=None, ws=None):
        """One query for each sequence: row b of ``q`` attends to the first seq_lens[b] cached rows of sequence b.
        Where plan_batch packs tokens of a batch with idle sequences in between, gather them by sequence first."""
        B = q.shape[0]
        c = self.cfg
        if o_out is None:
            o_out = torch.empty(B, c.n_heads * c.d_h, dtype=self.dtype, device=q.device)
        nb = L.gmla_decode_workspace_size(c, B)
        if ws is None and self.block_scaled:
            stream = _stream_of(q)
            c = self._status_cfg(q.device)
            with self._scratch.lock:
                ws = self._scratch.get("decode", nb, q.device, stream)
                L.check(L.gmla_decode(c, self.w, _p(q), _p(gate_logits), self.cache_arg(cache, q.device), _p(seq_lens),
                                      B, _p(o_out), ws.data_ptr(), ws.numel(), stream), "gmla_decode")
            return o_out
        if ws is None:
            ws = self.workspace("decode", nb, q.device)
        L.check(L.gmla_decode(c, self.w, _p(q), _p(gate_logits), self.cache_arg(cache, q.device), _p(seq_lens), B,
                              _p(o_out), ws.data_ptr(), ws.numel(), self._stream()), "gmla_decode")
        return o_out

    def prefill(self, q, gate_logits, cache: LatentCache, cu_seqlens, max_seqlen: int, o_out=None):
        T = q.shape[0]
        B = cu_seqlens.shape[0] - 1
        c = self.cfg
        if o_out is None:
            o_out = torch.empty(T, c.n_heads * c.d_h, dtype=self.dtype, device=q.device)
        nb = L.gmla_prefill_workspace_size(c, T, B)
        ws = self.workspace("prefill", nb, q.device)
        L.check(L.gmla_prefill(c, self.w, _p(q), _p(gate_logits), cache.struct(), _p(cu_seqlens), B, T,
                               int(max_seqlen), _p(o_out), ws.data_ptr(), ws.numel(), self._stream()),
                "gmla_prefill")
        return o_out

    def gate_out(self, o, gate_logits=None, y_out=None):
        T = o.shape[0]
        c = self.cfg
        if y_out is None:
            y_out = torch.empty(T, c.d_model, dtype=self.dtype, device=o.device)
        nb = L.gmla_gate_out_workspace_size(c, T)
        ws = self.workspace("gate_out", nb, o.device)
        L.check(L.gmla_gate_out(c, self.w, _p(o), T, _p(gate_logits), _p(y_out), ws.data_ptr(), ws.numel(),
                                self._stream()), "gmla_gate_out")
        return y_out

    def cache_append(self, latents, cu_seqlens, seq_lens, cache: LatentCache) -> None:
        """Append the new latent rows [T, d_c] (packed by sequence, rows may be strided) to a
        block-scaled cache: sequence b's rows cu_seqlens[b] .. cu_seqlens[b + 1] - 1 go to its
        last positions, seq_lens[b] (the new rows included) being its length afterwards."""
        stream = _stream_of(latents)
        dev, c = latents.device, self.cfg
        B = seq_lens.shape[0]
        if latents.dim() != 2:
            raise ValueError("latents is [T, d_c]")
        T = latents.shape[0]
        _check(latents, "latents", self.dtype, (T, c.d_c), dev)
        _check(seq_lens, "seq_lens", torch.int32, (B,), dev)
        _check(cu_seqlens, "cu_seqlens", torch.int32, (B + 1,), dev)
        if latents.stride(1) != 1:
            raise ValueError("latents: the elements of a row must be contiguous")
        ws = self._status.word("layer", dev)
        L.check(L.gmla_cache_append(c, self._cache_struct(cache, dev), latents.data_ptr(),
                                    latents.stride(0) if T > 1 else c.d_c, _p(cu_seqlens), _p(seq_lens), B, T,
                                    ws.data_ptr(), ws.numel(), stream), "gmla_cache_append")

    def _cache_struct(self, cache: LatentCache, device) -> L.gmla_cache:
        """The cache argument of a block-scaled layer."""
        if cache.scales is None:
            raise ValueError("a block-scaled layer needs a cache with scales")
        if cache.data.device != device or cache.data.element_size() != 1 or cache.data.shape[-1] != self.row:
            raise ValueError(f"a block-scaled cache holds 1-byte codes in rows of {self.row} on {device}")
        return cache.struct()

    def cache_arg(self, cache: LatentCache, device) -> L.gmla_cache:
        """The cache argument of a decode (without scales a block-scaled layer's is left to the library to refuse)."""
        return self._cache_struct(cache, device) if self.block_scaled and cache.scales is not None else cache.struct()

    def _project_and_append(self, x, cache, q_out, gate_logits, cu_seqlens, seq_lens):
        if cu_seqlens is None or seq_lens is None:
            raise ValueError("a block-scaled cache needs cu_seqlens and seq_lens")
        stream = _stream_of(x)
        T, dev = x.shape[0], x.device
        cfg = self._status_cfg(dev, staging=True)      # over a bf16 cache of one sequence, row t the latent of token t
        if cfg.d_rope:
            raise ValueError("a block-scaled cache covers NoPE")
        if q_out is None:
            q_out = torch.empty(T, cfg.n_heads, cfg.d_h, dtype=self.dtype, device=dev)
        if gate_logits is None:
            gate_logits = torch.empty(T, self.G, dtype=torch.float32, device=dev)
        rows = torch.empty(max(T, 1), cfg.d_c, dtype=self.dtype, device=dev)
        staging = LatentCache(rows.view(1, max(T, 1), cfg.d_c))
        order = torch.arange(T, dtype=torch.int32, device=dev)
        slot = torch.zeros(T, dtype=torch.int32, device=dev)
        with self._scratch.lock:
            ws = self._scratch.get("project", L.gmla_latent_project_workspace_size(cfg, T), dev, stream)
            L.check(L.gmla_latent_project(cfg, self.w, _p(x), T, _p(order), _p(slot), staging.struct(), _p(q_out),
                                          _p(gate_logits), ws.data_ptr(), ws.numel(), stream), "gmla_latent_project")
        self.cache_append(rows[:T], cu_seqlens, seq_lens, cache)
        return q_out, gate_logits

    def gate_out_w4(self, o, w4: W4Weight, gate_logits=None, y_out=None):
        """gate_out with W_o in 4 bits (``w4`` is [d_model, H*d_h])."""
        stream = _stream_of(o)
        dev, T = o.device, o.shape[0]
        c = self._status_cfg(dev)
        K = c.n_heads * c.d_h
        _check(o, "o", self.dtype, (T, K), dev)
        if w4.group not in (32, 64, 128) or K % w4.group:
            raise ValueError("w4.group must be 32, 64 or 128 and divide H*d_h")
        _check(w4.codes, "w4.codes", torch.uint8, (c.d_model, K // 2), dev)
        _check(w4.scales, "w4.scales", torch.bfloat16, (c.d_model, K // w4.group), dev)
        if gate_logits is not None:
            _check(gate_logits, "gate_logits", torch.float32, (T, self.G), dev)
        if y_out is None:
            y_out = torch.empty(T, c.d_model, dtype=self.dtype, device=dev)
        else:
            _check(y_out, "y_out", self.dtype, (T, c.d_model), dev)
        with self._scratch.lock:
            ws = self._scratch.get("gate_out_w4", L.gmla_gate_out_w4_workspace_size(c, T), dev, stream)
            L.check(L.gmla_gate_out_w4(c, w4.struct(), _p(o), T, _p(gate_logits), _p(y_out), ws.data_ptr(), ws.numel(),
                                       stream), "gmla_gate_out_w4")
        return y_out

    def sync_status(self):
        """Synchronise and raise if any kernel of the layer's calls, captured ones included, reported a
        device-side fault. The report stays until clear_status."""
        self._status.sync_status()
        for key, ws in self._ws.items():
            L.check(L.gmla_sync_status(ws.data_ptr(), self._stream()), f"device status ({key})")

    def clear_status(self):
        """Synchronise and forget what the layer's calls have reported."""
        self._status.clear_status()
        for ws in self._ws.values():
            L.check(L.gmla_clear_status(ws.data_ptr(), self._stream()), "clear_status")

    # -- whole steps
    def decode_step(self, x, cache: LatentCache, seq_lens, positions, seq_ids, *, cu_seqlens=None,
                    w4: Optional[W4Weight] = None):
        """One decode step: project (writing each new latent row), attend, gate, W_o (in 4
        bits when ``w4`` is given). Row b of ``x`` is sequence b's token: sequences that get none in this
        step come last (``decode`` takes row b of its queries as sequence b's). A block-scaled cache
        needs the step's ``cu_seqlens``."""
        if self.block_scaled:
            q, g = self.latent_project(x, positions, seq_ids, cache, cu_seqlens=cu_seqlens, seq_lens=seq_lens)
        else:
            q, g = self.latent_project(x, positions, seq_ids, cache)
        o = self.decode(q, g, cache, seq_lens)
        return self.gate_out(o) if w4 is None else self.gate_out_w4(o, w4)

    def prefill_step(self, x, cache: LatentCache, cu_seqlens, max_seqlen, positions, seq_ids):
        q, g = self.latent_project(x, positions, seq_ids, cache)
        o = self.prefill(q, g, cache, cu_seqlens, max_seqlen)
        return self.gate_out(o)
