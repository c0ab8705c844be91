"""The rotary positions and the paged cache in 64 bits on the CPU, row by row, written from the definitions; shared by
the tests of both."""
import math

import torch


def turn(x, pos, freqs, interleaved=False, amplitude=1.0, inverse=False):
    """x [..., d] float64, pos broadcastable to x's leading dimensions, freqs a list of radians per position."""
    y = x.clone()
    rot = 2 * len(freqs)
    t = pos.double()[..., None] * torch.tensor(freqs, dtype=torch.float64)
    c, s = amplitude * torch.cos(t), amplitude * torch.sin(t)
    if inverse:
        s = -s
    i = torch.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def quantise(x):
    """x [..., d] of a 16-bit type: codes (int64) and (scale, mid) float16, by the formula (fp32, as it says)."""
    g = x.float().unflatten(-1, (-1, 32))
    lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    scale = ((hi - lo) / torch.tensor(15.0)).half()
    mid = (lo + 8 * scale.float()).half()
    c = ((g - mid.float()) / scale.float()).round() + 8
    c = torch.where(scale > 0, c, torch.full_like(c, 8.0)).clamp(0, 15)
    return c.long().flatten(-2), torch.cat([scale, mid], -1)


def place(d, is_k):
    """Where value e's code is in a row: nibble index (byte 2n: low, 2n+1: high), for e = 0 .. d-1."""
    n = d // 32
    at = []
    for e in range(d):
        g, i = divmod(e, 32)
        if is_k:
            c, j = divmod(i, 8)
            at.append(8 * (c * n + g) + j)
        else:
            r, j = divmod(i, 4)
            at.append(4 * (r * n + g) + j)
    return torch.tensor(at)


def pack(codes, is_k):
    d = codes.shape[-1]
    nib = torch.zeros_like(codes)
    nib[..., place(d, is_k)] = codes
    return (nib[..., 0::2] + 16 * nib[..., 1::2]).to(torch.uint8)


def unpack(rows, is_k):
    r = rows.long()
    nib = torch.stack([r % 16, r // 16], -1).flatten(-2)
    return nib[..., place(nib.shape[-1], is_k)]


def values(rows, par, is_k):
    """Rows of a 4-bit cache in 64 bits, and the parts scale (c - 8) of them."""
    c = (unpack(rows, is_k).double() - 8).unflatten(-1, (-1, 32))
    part = par[..., :1].double() * c
    return (part + par[..., 1:].double()).flatten(-2), part.flatten(-2)


def key_set(p, r, dil, globals_):
    keys = {p - dil * t for t in range(min(r, p // dil) + 1)}
    if globals_ is not None:
        g = set(int(x) for x in globals_)
        if p in g:
            return list(range(p + 1))
        keys |= {x for x in g if 0 <= x <= p}
    return sorted(keys)


def attend(q, cache, table, rows, r, dil, globals_, scale):
    """y [N, Hq, d] float64 (NaN where a row is none), the sums p |v| by which its rounding errors are bounded, and the
    largest sum of the |terms| of a finite score.  rows: (sequence, position) or None each; cache: CPU (k, v, k_par, v_par); pages outside the cache hold no keys."""
    k, v, k_par, v_par = cache
    pages, hkv, page = k.shape[:3]
    N, hq, d = q.shape
    y = torch.full((N, hq, d), math.nan, dtype=torch.float64)
    by, big = torch.zeros_like(y), 0.0
    for n, at in enumerate(rows):
        if at is None:
            continue
        s, p = at
        for h in range(hkv):
            keys = key_set(p, r, dil[h], None if globals_ is None else globals_[s])
            where = [(int(table[s, j // page]), j % page) for j in keys]
            where = [w for w in where if 0 <= w[0] < pages]
            heads = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            if not where:
                y[n, heads] = 0
                continue
            a = torch.tensor([w[0] for w in where])
            b = torch.tensor([w[1] for w in where])
            if k_par is None:
                kk, vv = k[a, h, b].double(), v[a, h, b].double()
                size = kk.abs()
            else:
                kk, size = values(k[a, h, b], k_par[a, h, b], True)
                size = size.abs() + (kk - size).abs()
                vv = values(v[a, h, b], v_par[a, h, b], False)[0]
            size = q[n, heads].double().abs() @ size.T * abs(scale)
            big = max(big, size[torch.isfinite(size)].max().item())
            w = torch.softmax(q[n, heads].double() @ kk.T * scale, -1)
            y[n, heads], by[n, heads] = w @ vv, w @ vv.abs()
    return y, by, big


def attend_tolerance(y, by, big, dtype, bits):
    """Half a step for each rounding, relative to the sum of p |v|: over 16 bits P as two bf16 parts (2^-15) or two
    f16 ones (2^-20); over 4 bits V as f16 (2^-11), and P as f16 with bf16 queries (another 2^-11) or as two f16 parts (2^-20);
    and the output.  In fp32: a score is off by at most about 32 steps of 2^-24 of the sum of its |terms| `big` (8
    accumulations that may truncate, the group sums, the scaling), which moves P by that share, and so does its base's
    share the sum; exponentials and sums of P, and the 1024 times larger sums of 4-bit codes: 2^-12 in all."""
    u = torch.finfo(dtype).eps / 2
    half = dtype == torch.float16
    p = (2.0 ** -20 if half else 2.0 ** -15) if bits == 16 else (2.0 ** -11 + 2.0 ** -20 if half else 2.0 ** -10)
    return p * by + u * y.abs() + (2.0 ** -12 + 2.0 ** -18 * big) * (by + y.abs()) + 1e-7
