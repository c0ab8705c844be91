"""Rotary positions for q and k (``lf_attn_rotary``): in front of ``lf_attn.fwd`` and, transposed, behind
``lf_attn.bwd``.

``fwd`` takes q, k, v as views [B, heads, T, d] of any strides (of one packed projection, say) and gives the
contiguous [B, heads, T, d] rows that the attention reads; ``bwd`` takes the attention's gradients back, into views
of a packed gradient where ``out`` names them.  Work runs in the library's kernels only.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
from typing import Optional, Sequence

import torch

from . import lf_attn
from .lf_attn import LfAttnError, _dtype_code, _ptr


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


def _on(stream: Optional[torch.cuda.Stream], tensors):
    """The tensors' device, and ``stream`` (default: the device's current one) as the current stream: what is
    allocated within belongs to that stream, and tensors of another one are marked as used by it."""
    device = tensors[0].device
    if device.type != "cuda":
        raise ValueError("tensors must be on a CUDA device")
    if any(t.device != device for t in tensors):
        raise ValueError("all tensors must be on one device")
    stack = contextlib.ExitStack()
    stack.enter_context(torch.cuda.device(device))
    if stream is not None:
        if stream.device != device:
            raise ValueError("the stream is of another device than the tensors")
        if stream != torch.cuda.current_stream(device):
            if not torch.cuda.is_current_stream_capturing():
                for t in tensors:
                    t.record_stream(stream)
            stack.enter_context(torch.cuda.stream(stream))
    return stack, ctypes.c_void_p((stream or torch.cuda.current_stream(device)).cuda_stream)


def _check_freqs(f: Optional[torch.Tensor], d: int) -> int:
    if f is None:
        return 0
    if f.dtype != torch.float64 or f.dim() != 1 or not f.is_contiguous():
        raise ValueError("freqs must be a contiguous float64 [rot / 2] tensor")
    if 2 * f.numel() > d:
        raise ValueError("rot = 2 * len(freqs) must not exceed the head dimension")
    return 2 * f.numel()


def _turn(q, k, v, f, pos, interleaved, amplitude, out, out_dtype, stream, inverse):
    rows = [q, k, v]
    have = [t for t in rows if t is not None]
    if not have:
        raise ValueError("one of q, k and v must be given")
    first = have[0]
    if any(t.dim() != 4 for t in have):
        raise ValueError("q, k, v must be [B, heads, T, d]")
    B, _, T, d = first.shape
    if any((t.shape[0], t.shape[2], t.shape[3]) != (B, T, d) for t in have):
        raise ValueError("q, k, v must share B, T and d")
    if k is not None and v is not None and k.shape[1] != v.shape[1]:
        raise ValueError("k and v must have the same heads")
    if any(t.dtype != first.dtype for t in have):
        raise TypeError("q, k, v must share a dtype")
    rot = _check_freqs(f, d)
    if pos is not None and (pos.dtype != torch.int32 or tuple(pos.shape) not in ((T,), (B, T)) or
                            (T > 1 and pos.stride(-1) != 1)):
        raise ValueError("pos must be an int32 [T] or [B, T] tensor with its last dimension contiguous")
    if out is not None:
        out = list(out)
        if len(out) != 3:
            raise ValueError("out must name three tensors (None for absent ones)")
        for t, o in zip(rows, out):
            if (t is None) != (o is None) or (t is not None and o.shape != t.shape):
                raise ValueError("out must have the shapes of q, k, v")
        od = [o.dtype for o in out if o is not None]
        if any(x != od[0] for x in od) or (out_dtype is not None and out_dtype != od[0]):
            raise TypeError("out must share one dtype")
        out_dtype = od[0]
    out_dtype = out_dtype or first.dtype
    codes = _dtype_code(first), _dtype_code(torch.empty(0, dtype=out_dtype))
    for t in have + [o for o in out or [] if o is not None]:
        if t.shape[3] > 1 and t.stride(3) != 1:
            raise ValueError("the d values of a row must be contiguous")
    used = have + [t for t in (f, pos) if t is not None] + [o for o in out or [] if o is not None]
    stack, s = _on(stream, used)
    with stack:
        if out is None:
            out = [None if t is None else torch.empty(t.shape, dtype=out_dtype, device=t.device) for t in rows]
        if all(t.numel() == 0 for t in have):  # nothing to turn: empty tensors have no address
            return tuple(out)
        strides = (ctypes.c_int64 * 18)(*[0 if t is None else t.stride(i) for t in rows + out for i in range(3)])
        st = lf_attn.load().lf_attn_rotary(
            *[_ptr(t) for t in rows + out], strides, B, q.shape[1] if q is not None else 0,
            next((t.shape[1] for t in (k, v) if t is not None), 0), T, d, _ptr(pos),
            pos.stride(0) if pos is not None and pos.dim() == 2 else 0, _ptr(f) if rot else None, rot,
            1 if interleaved else 0, 1 if inverse else 0, float(amplitude), codes[0], codes[1], s)
    if st != 0:
        raise LfAttnError(st, "lf_attn_rotary")
    return tuple(out)


def fwd(q: Optional[torch.Tensor], k: Optional[torch.Tensor] = None, v: Optional[torch.Tensor] = None, *,
        freqs: Optional[torch.Tensor], pos: Optional[torch.Tensor] = None, interleaved: bool = False,
        amplitude: float = 1.0, out=None, out_dtype: Optional[torch.dtype] = None,
        stream: Optional[torch.cuda.Stream] = None):
    """(q, k, v) with q and k turned by their positions and v copied, each [B, heads, T, d] and contiguous unless
    ``out`` gives the three tensors to write.  ``pos``: int32 [T] or [B, T] (default 0 .. T-1).  Pairs are
    (i, i + rot / 2), or (2i, 2i + 1) when ``interleaved``.  ``out_dtype`` may be a 16-bit type for fp32 rows."""
    return _turn(q, k, v, freqs, pos, interleaved, amplitude, out, out_dtype, stream, False)


def bwd(dq: Optional[torch.Tensor], dk: Optional[torch.Tensor] = None, dv: Optional[torch.Tensor] = None, *,
        freqs: Optional[torch.Tensor], pos: Optional[torch.Tensor] = None, interleaved: bool = False,
        amplitude: float = 1.0, out=None, out_dtype: Optional[torch.dtype] = None,
        stream: Optional[torch.cuda.Stream] = None):
    """The gradients of fwd's q, k, v from those of its outputs (the transpose: turned by the negative angle), for
    instance lf_attn.bwd's fp32 ones into the 16-bit views ``out`` of a packed gradient."""
    return _turn(dq, dk, dv, freqs, pos, interleaved, amplitude, out, out_dtype, stream, True)
