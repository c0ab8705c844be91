"""The paged key/value cache, of 16 or of 4 bits, and the attention of new tokens over it (``lf_attn_cache_*``).

One step of a model that answers token by token:

    plan = Plan(cache, table, cu_tokens, context, n_tokens, q_heads, r, ...)   # once a step, for all layers
    q = append(cache, plan, k, v, q=q, freqs=freqs)                            # per layer: keys turned on the way
    y = fwd(cache, plan, q)

``table``, ``cu_tokens``, ``context`` and ``global_idx`` stay on the device, and ``Plan.refresh`` lays the step out
again from what they then hold, so a step can be captured into a CUDA graph and replayed.  Work runs in the library's
kernels only.
"""
from __future__ import annotations

import struct
from typing import Optional

import torch

from . import lf_attn
from .lf_attn import LF_BF16, LF_F16, LfAttnError, _dil_array, _ptr
from .rotary import _check_freqs, _on_stream

_PACK4, _PACK12 = struct.Struct("4q").pack, struct.Struct("12q").pack
_CODES = {torch.bfloat16: LF_BF16, torch.float16: LF_F16}
_MOST = (1 << 31) - 1


def _int32(t: torch.Tensor, shape, what: str) -> torch.Tensor:
    if t.dtype != torch.int32 or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError("%s must be a contiguous int32 %s tensor" % (what, list(shape)))
    return t


class KVCache:
    """The pages of one layer.  16 bits: k, v [pages, kv_heads, page, d] (bfloat16 or float16).  4 bits: k, v
    [pages, kv_heads, page, d / 2] uint8 codes and k_par, v_par [pages, kv_heads, page, d / 32, 2] float16 (scale,
    mid) of each group of 32 values, in the order that ``include/lf_attn.h`` describes."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_par: Optional[torch.Tensor] = None,
                 v_par: Optional[torch.Tensor] = None):
        if k.dim() != 4 or v.shape != k.shape or v.dtype != k.dtype:
            raise ValueError("k and v must be [pages, kv_heads, page, width] of one dtype")
        if (k_par is None) != (v_par is None):
            raise ValueError("k_par and v_par go together")
        self.pages, self.kv_heads, self.page, width = k.shape
        self.bits = 16 if k_par is None else 4
        self.d = width if self.bits == 16 else 2 * width
        if self.bits == 16 and k.dtype not in (torch.bfloat16, torch.float16):
            raise TypeError("a 16-bit cache is bfloat16 or float16")
        if self.bits == 4:
            shape = (self.pages, self.kv_heads, self.page, self.d // 32, 2)
            if k.dtype != torch.uint8:
                raise TypeError("the codes of a 4-bit cache are uint8")
            for t in (k_par, v_par):
                if t.dtype != torch.float16 or tuple(t.shape) != shape:
                    raise ValueError("k_par and v_par must be float16 %s" % list(shape))
        for t in (k, v, k_par, v_par):
            if t is not None and (not t.is_contiguous() or t.device != k.device):
                raise ValueError("the cache's tensors must be contiguous and on one device")
        self.k, self.v, self.k_par, self.v_par = k, v, k_par, v_par
        self.shape, self.device_index = (self.kv_heads, self.page, self.d, self.bits), k.get_device()

    @classmethod
    def empty(cls, pages: int, kv_heads: int, page: int, d: int, dtype: torch.dtype = torch.bfloat16, bits: int = 16,
              device="cuda") -> "KVCache":
        """A cache whose pages hold nothing yet.  ``dtype`` counts for 16 bits only."""
        if bits == 16:
            return cls(*[torch.empty(pages, kv_heads, page, d, dtype=dtype, device=device) for _ in range(2)])
        if bits != 4 or d % 32:
            raise ValueError("bits must be 16 or 4, and d a multiple of 32")
        codes = [torch.empty(pages, kv_heads, page, d // 2, dtype=torch.uint8, device=device) for _ in range(2)]
        par = [torch.empty(pages, kv_heads, page, d // 32, 2, dtype=torch.float16, device=device) for _ in range(2)]
        return cls(*codes, *par)


class Plan:
    """One step over caches shaped as ``cache``: rows [cu_tokens[s], cu_tokens[s+1]) of the step's n_tokens rows are
    sequence s's new tokens, at positions context[s] on; rows behind the last sequence are no tokens.  ``table``:
    int32 [n_seqs, max_pages]; ``global_idx``: int32 [n_seqs, n_global], any order; ``dil``: an int or one per kv head;
    ``r``: how many (dilated) positions back a token sees beside the global ones, None for all of them.

    ``table`` is read when append and fwd run, the other tensors when the plan is made or refreshed."""

    def __init__(self, cache: KVCache, table: torch.Tensor, cu_tokens: torch.Tensor, context: torch.Tensor,
                 n_tokens: int, q_heads: int, r: Optional[int] = None, dil=None,
                 global_idx: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
        if context.dim() != 1 or table.dim() != 2:
            raise ValueError("context must be [n_seqs] and table [n_seqs, max_pages]")
        S = context.shape[0]
        self.n_seqs, self.n_tokens, self.q_heads, self.kv_heads = S, int(n_tokens), int(q_heads), cache.kv_heads
        if not 0 <= self.n_tokens <= _MOST or not 1 <= self.q_heads <= _MOST:
            raise ValueError("n_tokens must not be negative and q_heads at least 1, both in 32 bits")
        self.page, self.max_pages = cache.page, table.shape[1]
        # the library's sizes have 32 bits; past them a window is all of a sequence, and a dilation past its length
        self.r = _MOST if r is None else min(int(r), _MOST)
        if self.r < 0:
            raise ValueError("r must not be negative")
        if dil is not None:
            dil = [dil] * cache.kv_heads if isinstance(dil, int) else [int(x) for x in dil]
            if min(dil, default=1) < 1:
                raise ValueError("dil must be at least 1")
            dil = [min(x, _MOST) for x in dil]
        self.dil = _dil_array(dil, cache.kv_heads)
        self.table = _int32(table, (S, self.max_pages), "table")
        self.cu_tokens = _int32(cu_tokens, (S + 1,), "cu_tokens")
        self.context = _int32(context, (S,), "context")
        self.n_global = 0 if global_idx is None else global_idx.shape[1]
        self.global_idx = None
        if self.n_global:
            self.global_idx = _int32(global_idx, (S, self.n_global), "global_idx")
        size = lf_attn.load().lf_attn_cache_plan_bytes(S, self.n_tokens, self.n_global)
        if size == 0:
            raise LfAttnError(1, "lf_attn_cache_plan_bytes")
        self.d, self.bits, self.shape = cache.d, cache.bits, cache.shape
        self.workspace_bytes = lf_attn.load().lf_attn_cache_workspace_bytes(
            self.n_tokens, self.n_global, self.page, self.max_pages, self.q_heads, self.kv_heads, self.d, self.bits,
            self.r)
        self.device_index = context.get_device()

        def make(raw):
            self._streams = {raw}
            return torch.empty(size, dtype=torch.uint8, device=context.device)

        self.buffer = _on_stream(stream, self.device_index, self._inputs(), make)
        self.refresh(stream)

    def _inputs(self):
        return self.cu_tokens, self.context, self.table, self.global_idx

    def _used_by(self, raw):
        """The buffer, which only the plan holds, outlives the plan until the work of every stream that read it is done."""
        if raw not in self._streams and not torch.cuda.is_current_stream_capturing():
            self.buffer.record_stream(torch.cuda.current_stream(self.device_index))
            self._streams.add(raw)

    def refresh(self, stream: Optional[torch.cuda.Stream] = None) -> "Plan":
        """Lays the step out again, from what cu_tokens, context and global_idx hold when the call runs."""
        def call(raw):
            self._used_by(raw)
            st = lf_attn.load().lf_attn_cache_plan(
                _ptr(self.cu_tokens), _ptr(self.context), self.n_seqs, self.n_tokens, _ptr(self.global_idx),
                self.n_global, self.page, self.max_pages, self.q_heads, self.kv_heads, self.d, self.bits,
                self.r, self.dil,
                _ptr(self.buffer), raw)
            if st != 0:
                raise LfAttnError(st, "lf_attn_cache_plan")

        _on_stream(stream, self.context.get_device(), (*self._inputs(), self.buffer), call)
        return self

    def _check(self, cache: KVCache):
        if cache.shape != self.shape:
            raise ValueError("the plan was made for a cache with other heads, pages or bits")
        if cache.device_index != self.device_index:
            raise ValueError("plan and cache must be on one device")


def _rows(t: torch.Tensor, n: int, heads: int, d: int, dtype, what: str):
    """The (token, head) strides of rows t, checked."""
    if t.shape != (n, heads, d):
        raise ValueError("%s must be [n_tokens, heads, d] = %s" % (what, [n, heads, d]))
    if t.dtype is not dtype:
        raise TypeError("%s must be %s" % (what, dtype))
    a, b, c = t.stride()
    if c != 1:
        raise ValueError("the d values of a row of %s must be contiguous" % what)
    return a, b


def _code(cache: KVCache, dtype) -> int:
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError("rows must be bfloat16 or float16, got %s" % dtype)
    if cache.bits == 16 and dtype != cache.k.dtype:
        raise TypeError("rows and cache must share a dtype")
    return code


def _at(t):
    return None if t is None else t.data_ptr()


def append(cache: KVCache, plan: Plan, k: torch.Tensor, v: torch.Tensor, q: Optional[torch.Tensor] = None,
           freqs: Optional[torch.Tensor] = None, interleaved: bool = False, amplitude: float = 1.0,
           q_out: Optional[torch.Tensor] = None, held=None, stream: Optional[torch.cuda.Stream] = None):
    """Puts the step's keys (turned by their positions where ``freqs`` is given) and values into the cache, and gives
    the turned q (None without q).  k, v: [n_tokens, kv_heads, d], q: [n_tokens, q_heads, d], of any strides.

    ``held`` asks for what the cache now holds of these rows, as dense 16-bit rows (for 4 bits the dequantised
    values): True for new tensors, or the two to write; append then gives (q, k_held, v_held)."""
    plan._check(cache)
    dtype, n, hkv, d = k.dtype, plan.n_tokens, cache.kv_heads, cache.d
    code = _code(cache, dtype)
    strides = [*_rows(k, n, hkv, d, dtype, "k"), *_rows(v, n, hkv, d, dtype, "v"),
               *(_rows(q, n, plan.q_heads, d, dtype, "q") if q is not None else (0, 0))]
    if q_out is not None:
        if q is None:
            raise ValueError("q_out without q")
        _rows(q_out, n, plan.q_heads, d, dtype, "q_out")
    hk = hv = None
    if held is not None and held is not False and held is not True:
        if len(held) != 2:
            raise ValueError("held must be True or the two tensors to write")
        hk, hv = held
        for t in held:
            _rows(t, n, hkv, d, dtype, "held")
    rot = _check_freqs(freqs, d)
    used = (k, v, q, freqs, q_out, hk, hv)
    if stream is not None:
        used += (plan.buffer, plan.table, cache.k, cache.v, cache.k_par, cache.v_par)

    def call(raw):
        nonlocal q_out, hk, hv
        new = lambda t: torch.empty_like(t, memory_format=torch.contiguous_format)  # noqa: E731
        if q is not None and q_out is None:
            q_out = new(q)
        if held is True:
            hk, hv = new(k), new(v)
        if n > 0:  # empty tensors have no address
            plan._used_by(raw)
            for t in (hk, hv, q_out):
                strides.extend((0, 0) if t is None else t.stride()[:2])
            st = lf_attn.load().lf_attn_cache_append(
                k.data_ptr(), v.data_ptr(), _at(q), _at(hk), _at(hv), _at(q_out), _PACK12(*strides), cache.k.data_ptr(),
                cache.v.data_ptr(), _at(cache.k_par), _at(cache.v_par), cache.pages, cache.page, plan.table.data_ptr(),
                plan.max_pages, plan.buffer.data_ptr(), plan.n_seqs, n, plan.n_global, plan.q_heads, hkv, d,
                freqs.data_ptr() if rot else None, rot, 1 if interleaved else 0, float(amplitude), code, cache.bits,
                raw)
            if st != 0:
                raise LfAttnError(st, "lf_attn_cache_append")
        return (q_out, hk, hv) if hk is not None else q_out

    return _on_stream(stream, cache.device_index, used, call)


def fwd(cache: KVCache, plan: Plan, q: torch.Tensor, scale: Optional[float] = None,
        out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
        stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The attention of the step's rows q [n_tokens, q_heads, d] over the cache, which already holds their own keys.
    Rows behind the last sequence are left as they are in ``out``.  ``workspace``: a uint8 tensor of
    ``plan.workspace_bytes`` (0: none is needed) for callers that keep one per stream."""
    plan._check(cache)
    n, heads, d, dtype = plan.n_tokens, plan.q_heads, cache.d, q.dtype
    code = _code(cache, dtype)
    qs = _rows(q, n, heads, d, dtype, "q")
    used = (q, out, workspace)
    if stream is not None:
        used += (plan.buffer, plan.table, cache.k, cache.v, cache.k_par, cache.v_par)
    if out is not None:
        _rows(out, n, heads, d, dtype, "out")
    if workspace is not None and (workspace.dtype != torch.uint8 or not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous uint8 tensor")

    def call(raw):
        y = torch.empty_like(q, memory_format=torch.contiguous_format) if out is None else out
        if n == 0:  # empty tensors have no address
            return y
        plan._used_by(raw)
        ws = workspace
        if ws is None and plan.workspace_bytes:
            ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device=q.device)
        st = lf_attn.load().lf_attn_cache_fwd(
            q.data_ptr(), y.data_ptr(), _PACK4(*qs, *y.stride()[:2]), cache.k.data_ptr(), cache.v.data_ptr(),
            _at(cache.k_par), _at(cache.v_par), cache.pages, cache.page, plan.table.data_ptr(), plan.max_pages,
            plan.buffer.data_ptr(), plan.n_seqs, n, plan.n_global, heads, cache.kv_heads, d, plan.r, plan.dil,
            d ** -0.5 if scale is None else float(scale), code, cache.bits, _at(ws), 0 if ws is None else ws.numel(), raw)
        if st != 0:
            raise LfAttnError(st, "lf_attn_cache_fwd")
        return y

    return _on_stream(stream, cache.device_index, used, call)
