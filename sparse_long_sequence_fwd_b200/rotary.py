"""Rotary positions for q and k (``lf_attn_rotary``): in front of ``lf_attn.fwd`` and, transposed, behind
``lf_attn.bwd``.

``fwd`` takes q, k, v as views [B, heads, T, d] of any strides (of one packed projection, say) and gives the
contiguous [B, heads, T, d] rows that the attention reads; ``bwd`` takes the attention's gradients back, into views
of a packed gradient where ``out`` names them.  Work runs in the library's kernels only.
"""
from __future__ import annotations

import math
import struct
from typing import Optional, Sequence

import torch

from . import lf_attn
from .lf_attn import LfAttnError


def freqs(rot: int, base: float = 10000.0, scaling: Optional[str] = None, factor: float = 1.0,
          trained: Optional[int] = None, turns: Sequence[float] = (1.0, 32.0), device=None) -> torch.Tensor:
    """Radians per position of the rot / 2 pairs, float64 on ``device``: base ** (-2 i / rot), stretched for
    contexts ``factor`` times as long:

    * ``"linear"``: every frequency / factor (position interpolation);
    * ``"base"``: the base is raised to base * factor ** (rot / (rot - 2)), so the first pair keeps its frequency and
      the last one is divided by factor;
    * ``"ramp"``: by parts (the YaRN method): a pair that makes over ``turns[1]`` turns in ``trained`` positions keeps
      its frequency, one that makes under ``turns[0]`` is divided by factor, those between are blended linearly.  The
      method goes with an amplitude of ``1 + 0.1 log(factor)`` (``amplitude`` of fwd).
    """
    if rot < 0 or rot % 2:
        raise ValueError("rot must be even and not negative")
    if not (base > 0 and factor > 0):
        raise ValueError("base and factor must be positive")
    if scaling not in (None, "linear", "base", "ramp"):
        raise ValueError("scaling must be None, 'linear', 'base' or 'ramp'")
    if scaling == "base":
        if rot < 4:
            raise ValueError("scaling 'base' needs rot >= 4")
        base = base * factor ** (rot / (rot - 2))
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        f = [x / factor for x in f]
    elif scaling == "ramp":
        if not trained or trained < 1 or not 0 < turns[0] < turns[1]:
            raise ValueError("scaling 'ramp' needs the trained length, and turns in rising order")
        out = []
        for x in f:
            keep = (trained * x / (2 * math.pi) - turns[0]) / (turns[1] - turns[0])
            keep = min(1.0, max(0.0, keep))
            out.append(x * keep + x / factor * (1 - keep))
        f = out
    return torch.tensor(f, dtype=torch.float64, device=device)


_PACK18 = struct.Struct("18q").pack
_CODES = {torch.float32: lf_attn.LF_F32, torch.bfloat16: lf_attn.LF_BF16, torch.float16: lf_attn.LF_F16}
_NONE = (0, 0, 0)


def _on_stream(stream: Optional[torch.cuda.Stream], index: int, tensors, call):
    """call(raw stream) with ``stream`` (default: the device's current one) as the current stream of device ``index``,
    which all of ``tensors`` (None: absent) must be on: what the call allocates belongs to that stream, and tensors are
    marked as used by a stream that is not the current one."""
    if index < 0:
        raise ValueError("tensors must be on a CUDA device")
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError("all tensors must be on one device")
    if stream is None:
        if torch._C._cuda_getDevice() == index:
            return call(torch._C._cuda_getCurrentRawStream(index))
        with torch.cuda.device(index):
            return call(torch._C._cuda_getCurrentRawStream(index))
    if stream.device.index != index:
        raise ValueError("the stream is of another device than the tensors")
    with torch.cuda.device(index):
        if stream != torch.cuda.current_stream() and not torch.cuda.is_current_stream_capturing():
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)
        with torch.cuda.stream(stream):
            return call(stream.cuda_stream)


def _check_freqs(f: Optional[torch.Tensor], d: int) -> int:
    if f is None:
        return 0
    if f.dtype is not torch.float64 or f.dim() != 1 or not f.is_contiguous():
        raise ValueError("freqs must be a contiguous float64 [rot / 2] tensor")
    rot = 2 * f.numel()
    if rot > d:
        raise ValueError("rot = 2 * len(freqs) must not exceed the head dimension")
    return rot


def _turn(q, k, v, f, pos, interleaved, amplitude, out, out_dtype, stream, inverse):
    first = q if q is not None else k if k is not None else v
    if first is None:
        raise ValueError("one of q, k and v must be given")
    if first.dim() != 4:
        raise ValueError("q, k, v must be [B, heads, T, d]")
    B, _, T, d = first.shape
    dtype = first.dtype
    in_code = _CODES.get(dtype)
    if in_code is None:
        raise TypeError("q, k, v must be float32, bfloat16 or float16, got %s" % dtype)
    rows, heads, strides, at = (q, k, v), [], [], []
    for t in rows:
        if t is None:
            heads.append(0)
            strides += _NONE
            at.append(None)
            continue
        if t.dim() != 4:
            raise ValueError("q, k, v must be [B, heads, T, d]")
        (b, h, n, e), (sb, sh, st, se) = t.shape, t.stride()
        if b != B or n != T or e != d:
            raise ValueError("q, k, v must share B, T and d")
        if t.dtype is not dtype:
            raise TypeError("q, k, v must share a dtype")
        if se != 1 and d > 1:
            raise ValueError("the d values of a row must be contiguous")
        heads.append(h)
        strides += (sb, sh, st)
        at.append(t.data_ptr())
    if heads[1] != heads[2] and k is not None and v is not None:
        raise ValueError("k and v must have the same heads")
    rot = _check_freqs(f, d)
    pos_at, pos_stride = None, 0
    if pos is not None:
        dims = pos.dim()
        if pos.dtype is not torch.int32 or not 1 <= dims <= 2 or pos.shape[-1] != T or (
                dims == 2 and pos.shape[0] != B) or (T > 1 and pos.stride(-1) != 1):
            raise ValueError("pos must be an int32 [T] or [B, T] tensor with its last dimension contiguous")
        if dims == 2:
            pos_stride = pos.stride(0)
        pos_at = pos.data_ptr()
    if out is None:
        out_dtype = out_dtype or dtype
        used = (q, k, v, f, pos)
    else:
        out = tuple(out)
        if len(out) != 3:
            raise ValueError("out must name three tensors (None for absent ones)")
        for t, o in zip(rows, out):
            if (t is None) != (o is None) or (t is not None and o.shape != t.shape):
                raise ValueError("out must have the shapes of q, k, v")
            if o is not None:
                out_dtype = out_dtype or o.dtype
                if o.dtype is not out_dtype:
                    raise TypeError("out must share one dtype")
                if d > 1 and o.stride(3) != 1:
                    raise ValueError("the d values of a row must be contiguous")
        used = (q, k, v, f, pos, *out)
    out_code = _CODES.get(out_dtype)
    if out_code is None:
        raise TypeError("out must be float32, bfloat16 or float16, got %s" % out_dtype)

    def call(raw):
        y = out
        if y is None:
            if out_dtype is dtype:
                y = tuple([None if t is None else torch.empty_like(t, memory_format=torch.contiguous_format)
                           for t in rows])
            else:
                y = tuple([None if t is None else
                           torch.empty_like(t, dtype=out_dtype, memory_format=torch.contiguous_format) for t in rows])
            n = T * d
            strides.extend((heads[0] * n, n, d, heads[1] * n, n, d, heads[2] * n, n, d))
        else:
            for t in y:
                strides.extend(_NONE if t is None else t.stride()[:3])
        if B == 0 or T == 0 or heads == [0, 0, 0]:  # nothing to turn: empty tensors have no address
            return y
        for t in y:
            at.append(None if t is None else t.data_ptr())
        st = lf_attn.load().lf_attn_rotary(
            *at, _PACK18(*strides), B, heads[0], heads[1] or heads[2], T, d, pos_at, pos_stride,
            f.data_ptr() if rot else None, rot, 1 if interleaved else 0, inverse, float(amplitude), in_code, out_code, raw)
        if st != 0:
            raise LfAttnError(st, "lf_attn_rotary")
        return y

    return _on_stream(stream, first.get_device(), used, call)


def fwd(q: Optional[torch.Tensor], k: Optional[torch.Tensor] = None, v: Optional[torch.Tensor] = None, *,
        freqs: Optional[torch.Tensor], pos: Optional[torch.Tensor] = None, interleaved: bool = False,
        amplitude: float = 1.0, out=None, out_dtype: Optional[torch.dtype] = None,
        stream: Optional[torch.cuda.Stream] = None):
    """(q, k, v) with q and k turned by their positions and v copied, each [B, heads, T, d] and contiguous unless
    ``out`` gives the three tensors to write.  ``pos``: int32 [T] or [B, T] (default 0 .. T-1).  Pairs are
    (i, i + rot / 2), or (2i, 2i + 1) when ``interleaved``.  ``out_dtype`` may be a 16-bit type for fp32 rows."""
    return _turn(q, k, v, freqs, pos, interleaved, amplitude, out, out_dtype, stream, 0)


def bwd(dq: Optional[torch.Tensor], dk: Optional[torch.Tensor] = None, dv: Optional[torch.Tensor] = None, *,
        freqs: Optional[torch.Tensor], pos: Optional[torch.Tensor] = None, interleaved: bool = False,
        amplitude: float = 1.0, out=None, out_dtype: Optional[torch.dtype] = None,
        stream: Optional[torch.cuda.Stream] = None):
    """The gradients of fwd's q, k, v from those of its outputs (the transpose: turned by the negative angle), for
    instance lf_attn.bwd's fp32 ones into the 16-bit views ``out`` of a packed gradient."""
    return _turn(dq, dk, dv, freqs, pos, interleaved, amplitude, out, out_dtype, stream, 1)
