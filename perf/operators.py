"""Rotary positions and the paged key/value cache of sparse attention, measured: the plain form of each operator in
elementary torch operations, and the framework's calls for the same work.

Operators
  rotary   q and k turned by their positions (and v beside them) from a packed projection [B, T, heads * d] into the
           contiguous [B, H, T, d] rows that the attention reads; its gradient takes fp32 [B, H, T, d] back to the packed form
  append   the new tokens' keys (turned on the way) and values into a paged cache of 16 or of 4 bits, and their turned queries
  attend   every new token's attention over the cache: its window (dilated per head) up to its own position, and the
           global tokens, each key once
  step     append, then attend: one layer of one decoding step

The turn: pair i of a row's first `rot` values, (x, y) -> a (x cos t - y sin t, y cos t + x sin t), t = position * freqs[i];
the pairs are (i, i + rot/2), or (2i, 2i+1) when interleaved; the values behind `rot` stay as they are.

A 4-bit cache holds groups of 32 values of a row as mid + scale (c - 8), c in 0..15, with scale and mid in fp16:
scale = (max - min) / 15, mid = min + 8 scale, c = (x - mid) / scale + 8 rounded to the nearest (ties to even), 8 where scale
is 0; x is the turned value rounded to the 16-bit type.  With n = d / 32 groups, the codes of a K row are 32-bit words [4][n],
word [c][g] holding values 32 g + 8 c + 0..7 from the lowest four bits up; those of a V row are 16-bit units [8][n], unit
[r][g] holding values 32 g + 4 r + 0..3.  k_par and v_par hold (scale, mid) of each group.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------- cases

def _rotary(name, back, dtype, B, T, hq, hkv, d, rot, pairs, factor):
    return {"name": name, "op": "rotary", "back": back, "dtype": dtype, "B": B, "T": T, "hq": hq, "hkv": hkv, "d": d,
            "rot": rot, "pairs": pairs, "factor": factor}


def _cache(name, op, dtype, bits, seqs, new, ctx, hq, hkv, d, page, r, dil, n_global, rot, pairs):
    return {"name": name, "op": op, "dtype": dtype, "bits": bits, "seqs": seqs, "new": new, "ctx": ctx, "hq": hq,
            "hkv": hkv, "d": d, "page": page, "r": r, "dil": dil, "n_global": n_global, "rot": rot, "pairs": pairs}


def listed():
    full = 1 << 20
    return [
        # training: the base layer's projection (12 heads of 64, 4096 tokens) turned before its attention
        _rotary("rotary_base", False, "bf16", 1, 4096, 12, 12, 64, 64, "half", 1.0),
        # ... and the fp32 gradients of two documents taken back to the projection's form
        _rotary("rotary_back_b2", True, "bf16", 2, 4096, 12, 12, 64, 64, "half", 1.0),
        # long documents: half of each head turned, interleaved, frequencies stretched four times; odd length
        _rotary("rotary_long_part", False, "f16", 1, 16383, 16, 8, 64, 32, "interleaved", 4.0),
        # prompts of three ragged lengths put into a 16-bit cache
        _cache("append_prompts", "append", "bf16", 16, 3, 4099, 0, 12, 12, 64, 64, 256, 1, 0, 64, "half"),
        # a long prompt put into a 4-bit cache
        _cache("append_prompt_4bit", "append", "bf16", 4, 1, 16384, 0, 16, 8, 64, 64, 256, 1, 0, 64, "half"),
        # one document, one new token: the base layer (window 256 back, one global token); latency counts
        _cache("attend_one_token", "attend", "bf16", 16, 1, 1, 4096, 12, 12, 64, 64, 256, 1, 1, 64, "half"),
        # a batch of dilated heads (every second key) at 8192 tokens
        _cache("attend_dilated", "attend", "f16", 16, 32, 32, 8192, 12, 12, 64, 16, 128, 2, 1, 64, "half"),
        # full attention, shared key heads of 128, ragged long sequences: the largest
        _cache("attend_full_shared", "attend", "bf16", 16, 16, 16, 32768, 32, 8, 128, 64, full, 1, 0, 128, "half"),
        # a batch over a 4-bit cache with a window and 32 global tokens
        _cache("attend_4bit_window", "attend", "bf16", 4, 64, 64, 16384, 12, 12, 64, 64, 256, 1, 32, 64, "half"),
        # few long sequences over a 4-bit cache, full attention
        _cache("attend_4bit_full", "attend", "bf16", 4, 4, 4, 65536, 32, 8, 128, 128, full, 1, 0, 128, "half"),
        # one decoding step of a layer: append and attend, 16 bits
        _cache("step_batch", "step", "bf16", 16, 48, 48, 4096, 12, 12, 64, 64, 256, 1, 1, 64, "half"),
        # ... and 4 bits, with shared heads and a few drafted tokens a sequence
        _cache("step_4bit", "step", "f16", 4, 8, 24, 8192, 16, 2, 128, 32, 1024, 1, 4, 64, "interleaved"),
    ]


def draw(rng):
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    op = rng.choice(["rotary", "rotary", "append", "append", "attend", "attend", "step"])
    d = rng.choice([64, 64, 128])
    hkv = rng.randint(1, 16)
    hq = hkv * rng.choice([1, 1, 2, 4, 5, 8])
    while hq > 64:
        hq -= hkv
    pairs = rng.choice(["half", "interleaved"])
    rot = rng.choice([d, d, d // 2, 2 * rng.randint(1, d // 2)])
    if op == "rotary":
        B, T = rng.randint(1, 3), log(1, 16384)
        while B * T * (hq + 2 * hkv) * d > 50_000_000:
            T = max(1, T // 2)
        c = _rotary("", rng.random() < 0.5, rng.choice(["bf16", "bf16", "f16", "f32"]), B, T, hq, hkv, d, rot, pairs,
                    rng.choice([1.0, 1.0, 8.0]))
    else:
        bits, page = rng.choice([16, 4]), rng.choice([8, 16, 32, 64, 128, 256])
        seqs = log(1, 64)
        r = rng.choice([0, log(1, 2048), log(1, 2048), 1 << 20])
        dil = rng.choice([1, 1, 2, 3]) if r < 1 << 20 else 1
        ctx = log(16, 32768)
        if op == "append":
            new = max(seqs, log(1, 16384))
            while new * (hq + 2 * hkv) * d > 50_000_000:
                new = max(1, new // 2)
            seqs, ctx = min(seqs, new), log(1, 2048)
        else:
            new = seqs * rng.choice([1, 1, 1, 2, 4])
        while seqs * ctx * hkv * d > 16 * 32768 * 8 * 128 or new * hkv * min(ctx, r + 64) * d > 16 * 32768 * 8 * 128:
            ctx = max(16, ctx // 2)
            if ctx == 16:
                break
        c = _cache("", op, rng.choice(["bf16", "bf16", "f16"]), bits, seqs, new, ctx, hq, hkv, d, page, r, dil,
                   rng.choice([0, 1, 1, 32]), rot, pairs)
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs

def _lengths(case):
    """New tokens and earlier tokens of each sequence, from the case alone: ragged, odd ones among them."""
    S, N, ctx = case["seqs"], case["new"], case["ctx"]
    new = [(i + 1) * N // S - i * N // S for i in range(S)]
    if S > 2 and N > 4 * S:  # a short and a long one
        take = new[0] - 1
        new[0], new[-1] = new[0] - take, new[-1] + take
    old = [ctx if S == 1 else max(0, ctx * (i + S) // (2 * S - 1) - i % 3) for i in range(S)]
    return new, old


def _freqs(case):
    rot = case["rot"]
    return [10000.0 ** (-2.0 * i / rot) / case.get("factor", 1.0) for i in range(rot // 2)]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = TYPES[case["dtype"]]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    heads = hq + 2 * hkv
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    s = {"case": case, "freqs": torch.tensor(_freqs(case), dtype=torch.float64, device="cuda"), "dt": dt}
    if case["op"] == "rotary":
        B, T = case["B"], case["T"]
        # positions of the batch: each sample at an offset of its own (a chunk of a longer document)
        start = torch.randint(0, 4096, (B, 1), generator=g, device="cuda", dtype=torch.int32)
        s["pos"] = (start + torch.arange(T, device="cuda", dtype=torch.int32)).contiguous()
        if case["back"]:
            s["grads"] = (randn(B, hq, T, d), randn(B, hkv, T, d), randn(B, hkv, T, d))
        else:
            s["qkv"] = randn(B, T, heads * d).to(dt)
        return s
    new, old = _lengths(case)
    S, N, page, bits = case["seqs"], sum(new), case["page"], case["bits"]
    order = torch.randperm(S, generator=g, device="cuda").tolist()
    new, old = [new[i] for i in order], [old[i] for i in order]
    longest = max(a + b for a, b in zip(new, old))
    per = -(-longest // page)
    need = [-(-(a + b) // page) for a, b in zip(new, old)]
    pages = sum(need) + 3
    where = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((S, per), -1, dtype=torch.int32)
    rows, at = where.cpu(), 0
    for i, n in enumerate(need):
        table[i, :n] = rows[at:at + n]
        at += n
    cu = torch.tensor([0] + new).cumsum(0).to(torch.int32)
    s["seq"] = torch.repeat_interleave(torch.arange(S), torch.tensor(new)).cuda()
    s["at"] = torch.cat([torch.arange(b, a + b) for a, b in zip(new, old)]).cuda()
    s["table"], s["cu"], s["context"] = table.cuda(), cu.cuda(), torch.tensor(old, dtype=torch.int32).cuda()
    s["qkv"] = randn(N, heads * d).to(dt)
    if bits == 16:
        s["k"], s["v"] = (torch.empty(pages, hkv, page, d, dtype=dt, device="cuda").normal_(generator=g) for _ in range(2))
        s["k_par"] = s["v_par"] = None
    else:
        s["k"], s["v"] = (torch.randint(0, 256, (pages, hkv, page, d // 2), generator=g, device="cuda", dtype=torch.uint8)
                          for _ in range(2))
        par = lambda: torch.stack([0.2 + 0.15 * torch.rand(pages, hkv, page, d // 32, generator=g, device="cuda"),  # noqa: E731
                                   0.3 * randn(pages, hkv, page, d // 32)], -1).half()
        s["k_par"], s["v_par"] = par(), par()
    s["glob"] = None
    if case["n_global"]:
        low = max(1, min(old))  # the global tokens lie in the earlier part of every sequence
        s["glob"] = torch.randint(0, low, (S, case["n_global"]), generator=g, device="cuda", dtype=torch.int32)
        s["glob"][:, 0] = 0
    # every head dilated but the first sixth, as in the dilated workload
    s["dil"] = [1 if h < hkv // 6 else case["dil"] for h in range(hkv)]
    if own:
        from sparse_long_sequence_fwd_b200 import kv_cache
        s["cache"] = kv_cache.KVCache(s["k"], s["v"], s["k_par"], s["v_par"])
        # made once per step, on the device, and shared by all layers of the step
        s["plan"] = kv_cache.Plan(s["cache"], s["table"], s["cu"], s["context"], N, hq, case["r"], dil=s["dil"],
                                  global_idx=s["glob"])
    return s


# ---------------------------------------------------------------- the plain forms

def _turn(x, pos, freqs, pairs, back=False):
    """x [..., d] in fp32, pos over x's leading dimensions: the turn (or its transpose) in fp32, its angles in 64 bits."""
    rot = 2 * freqs.numel()
    t = pos[..., None].double() * freqs
    cos, sin = t.cos().float(), t.sin().float()
    if back:
        sin = -sin
    if pairs == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


def _split(packed, case):
    """The q, k and v heads [..., heads, d] of a packed projection."""
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    x = packed.unflatten(-1, (hq + 2 * hkv, d))
    return x[..., :hq, :], x[..., hq:hq + hkv, :], x[..., hq + hkv:, :]


def _pack_k(c):
    n = c.shape[-1] // 32
    c = c.unflatten(-1, (n, 4, 8)).transpose(-3, -2)  # [c][g][8 values]
    return (c[..., 0::2] | c[..., 1::2] << 4).flatten(-3)


def _pack_v(c):
    n = c.shape[-1] // 32
    c = c.unflatten(-1, (n, 8, 4)).transpose(-3, -2)  # [r][g][4 values]
    return (c[..., 0::2] | c[..., 1::2] << 4).flatten(-3)


def _codes(packed, of_k):
    """[..., d/2] bytes -> [..., d] codes - 8 as whole numbers."""
    c = torch.stack([packed & 15, packed >> 4], -1).flatten(-2)
    n = c.shape[-1] // 32
    c = c.unflatten(-1, (4, n, 8) if of_k else (8, n, 4)).transpose(-3, -2).flatten(-3)
    return c.to(torch.int8) - 8


def _unpack(packed, par, of_k):
    c = _codes(packed, of_k).float().unflatten(-1, (-1, 32))
    par = par.float()
    return (par[..., 1:] + par[..., :1] * c).flatten(-2)


def _quantise(x):
    """x [..., d] in a 16-bit type: codes [..., d] (uint8) and (scale, mid) [..., d/32, 2]."""
    x = x.float().unflatten(-1, (-1, 32))
    low = x.amin(-1, keepdim=True)
    scale = ((x.amax(-1, keepdim=True) - low) / 15).half()
    mid = (low + 8 * scale.float()).half()
    c = torch.where(scale > 0, ((x - mid.float()) / scale.float()).round() + 8, torch.full_like(x, 8.0))
    return c.clamp(0, 15).to(torch.uint8).flatten(-2), torch.cat([scale, mid], -1)


def _append(s):
    case, dt = s["case"], s["dt"]
    q, k, v = _split(s["qkv"], case)
    at = s["at"][:, None]
    q = _turn(q.float(), at, s["freqs"], case["pairs"]).to(dt)
    k = _turn(k.float(), at, s["freqs"], case["pairs"]).to(dt)
    pages, slots = s["table"][s["seq"], s["at"] // case["page"]].long(), s["at"] % case["page"]
    if case["bits"] == 16:
        s["k"][pages, :, slots] = k
        s["v"][pages, :, slots] = v
        return q, k, v
    (ck, pk), (cv, pv) = _quantise(k), _quantise(v)
    s["k"][pages, :, slots], s["k_par"][pages, :, slots] = _pack_k(ck), pk
    s["v"][pages, :, slots], s["v_par"][pages, :, slots] = _pack_v(cv), pv
    held = lambda c, p: (p[..., 1:].float() + p[..., :1].float() * (c.float() - 8).unflatten(-1, (-1, 32))).flatten(-2).to(dt)  # noqa: E731
    return q, held(ck, pk), held(cv, pv)


def _keys(s):
    """The positions [N, Hkv, K] of every new token's keys, and which of them are keys (each once)."""
    case, p = s["case"], s["at"][:, None, None]
    dil = torch.tensor(s["dil"], device=p.device)[None, :, None]
    r = min(case["r"], int(s["table"].shape[1]) * case["page"])
    window = p - dil * torch.arange(r + 1, device=p.device)
    keep = window >= 0
    if s["glob"] is not None:
        g = s["glob"].long().sort(-1).values
        first = torch.cat([torch.ones_like(g[:, :1], dtype=torch.bool), g[:, 1:] != g[:, :-1]], -1)
        g, first = g[s["seq"]][:, None].expand(-1, case["hkv"], -1), first[s["seq"]][:, None]
        back = p - g
        inside = (back % dil == 0) & (back // dil <= r)
        window = torch.cat([window, g], -1)
        keep = torch.cat([keep, first & (back >= 0) & ~inside], -1)
    return window.clamp(min=0), keep


def _rows(s, j):
    case = s["case"]
    page = s["table"][s["seq"][:, None, None], j // case["page"]].long()
    head = torch.arange(case["hkv"], device=j.device)[None, :, None]
    return (page * case["hkv"] + head) * case["page"] + j % case["page"]


def _attend(s, q):
    case = s["case"]
    j, keep = _keys(s)
    rows = _rows(s, j)
    if case["bits"] == 16:
        k, v = s["k"].flatten(0, 2)[rows].float(), s["v"].flatten(0, 2)[rows].float()
    else:
        k = _unpack(s["k"].flatten(0, 2)[rows], s["k_par"].flatten(0, 2)[rows], True)
        v = _unpack(s["v"].flatten(0, 2)[rows], s["v_par"].flatten(0, 2)[rows], False)
    q = q.float().unflatten(1, (case["hkv"], -1))
    x = (q @ k.transpose(-1, -2)) * case["d"] ** -0.5
    x = x.masked_fill(~keep[:, :, None], -math.inf)
    p = (x - x.amax(-1, keepdim=True)).exp()
    y = (p @ v) / p.sum(-1, keepdim=True)
    return y.flatten(1, 2).to(s["dt"])


def _plain(s):
    case, dt = s["case"], s["dt"]
    if case["op"] == "rotary":
        pos = s["pos"][:, None]
        if case["back"]:
            dq, dk, dv = s["grads"]
            dq = _turn(dq, pos, s["freqs"], case["pairs"], True)
            dk = _turn(dk, pos, s["freqs"], case["pairs"], True)
            return torch.cat([dq, dk, dv], 1).transpose(1, 2).flatten(-2).to(dt)
        q, k, v = (x.transpose(1, 2).float() for x in _split(s["qkv"], case))
        q, k = _turn(q, pos, s["freqs"], case["pairs"]), _turn(k, pos, s["freqs"], case["pairs"])
        return q.to(dt), k.to(dt), v.to(dt).contiguous()
    q = _split(s["qkv"], case)[0]
    if case["op"] == "attend":
        return _attend(s, q)
    q, k, v = _append(s)
    y = (_attend(s, q),) if case["op"] == "step" else ()
    if case["bits"] == 16:
        return (q, s["k"], s["v"]) + y
    return (q, k, v) + y


# ---------------------------------------------------------------- the framework's calls

def _own(s):
    from sparse_long_sequence_fwd_b200 import kv_cache, rotary
    case = s["case"]
    inter = case["pairs"] == "interleaved"
    if case["op"] == "rotary":
        if case["back"]:
            dq, dk, dv = s["grads"]
            B, _, T, d = dq.shape
            packed = torch.empty(B, T, (case["hq"] + 2 * case["hkv"]) * d, dtype=s["dt"], device=dq.device)
            out = [x.transpose(1, 2) for x in _split(packed, case)]
            rotary.bwd(dq, dk, dv, freqs=s["freqs"], pos=s["pos"], interleaved=inter, out=out)
            return packed
        q, k, v = (x.transpose(1, 2) for x in _split(s["qkv"], case))
        return rotary.fwd(q, k, v, freqs=s["freqs"], pos=s["pos"], interleaved=inter)
    q, k, v = _split(s["qkv"], case)
    if case["op"] == "attend":
        return kv_cache.fwd(s["cache"], s["plan"], q)
    four = case["bits"] == 4
    got = kv_cache.append(s["cache"], s["plan"], k, v, q=q, freqs=s["freqs"], interleaved=inter, held=four)
    q = got[0] if four else got
    y = (kv_cache.fwd(s["cache"], s["plan"], q),) if case["op"] == "step" else ()
    return (tuple(got) if four else (q, s["k"], s["v"])) + y


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    es = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "rotary":
        n = case["B"] * case["T"]
        return {"bytes": n * (hq + 2 * hkv) * d * ((4 if case["back"] else es) + es) + n * 4,
                "flops": 3 * n * (hq + hkv) * case["rot"]}
    new, old = _lengths(case)
    N = sum(new)
    row = d * 2 if case["bits"] == 16 else d // 2 + d // 32 * 4  # bytes of one key's or value's row
    b = f = 0
    if case["op"] in ("append", "step"):
        b += N * (2 * hq + 2 * hkv) * d * 2 + N * 2 * hkv * row
        f += 3 * N * (hq + hkv) * case["rot"]
    if case["op"] in ("attend", "step"):
        b += 2 * N * hq * d * 2
        for n, c in zip(new, old):
            for h in range(hkv):
                dil = 1 if h < hkv // 6 else case["dil"]
                keys = [min(case["r"], p // dil) + 1 for p in range(c, c + n)]
                keys = [min(p + 1, x + case["n_global"]) for p, x in zip(range(c, c + n), keys)]
                # a sequence's tokens share their keys: each is read once
                reach = min(c + n, keys[-1] + (n - 1 if dil == 1 else sum(keys[:-1])))
                b += 2 * row * reach
                f += 4 * d * (hq // hkv) * sum(keys)
    return {"bytes": b, "flops": f}


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_turn(x, pos, case, sign=1.0):
    """x [..., d] float64 as complex numbers times exp(i t)."""
    f = torch.tensor(_freqs(case), dtype=torch.float64, device=x.device)
    t = sign * pos.double().unsqueeze(-1) * f
    e = torch.polar(torch.ones_like(t), t)
    y, rot = x.clone(), case["rot"]
    even, odd = (slice(0, rot // 2), slice(rot // 2, rot)) if case["pairs"] == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    z = torch.complex(x[..., even].contiguous(), x[..., odd].contiguous()) * e
    y[..., even], y[..., odd] = z.real, z.imag
    return y


def _exact_hold(x):
    """The values that the groups of x (a 16-bit type) are held as, in 64 bits."""
    x = x.double().reshape(*x.shape[:-1], -1, 32)
    low, high = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
    scale = ((high - low) / 15).half().double()
    mid = (low + 8 * scale).half().double()
    c = torch.nan_to_num((x - mid) / scale, nan=0.0).round().clamp(-8, 7)
    return (mid + scale * c).flatten(-2)


def _exact_cache(packed, par, units):
    """The values of a packed cache in 64 bits: each row is `units` x (d / 32) words of 32 / units values."""
    n, per = par.shape[-2], 32 // units
    byte = packed.long().reshape(*packed.shape[:-1], units, n, per // 2)
    word = (byte << (8 * torch.arange(per // 2, device=packed.device))).sum(-1)
    code = (word[..., None] >> (4 * torch.arange(per, device=packed.device))) % 16
    code = code.movedim(-2, -3).reshape(*packed.shape[:-1], n, 32).double()
    return (par[..., 1:].double() + par[..., :1].double() * (code - 8)).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    dt, hq, hkv, d = s["dt"], case["hq"], case["hkv"], case["d"]
    if case["op"] == "rotary":
        if case["back"]:
            g = [x.double() for x in s["grads"]]
            g = [_exact_turn(x, s["pos"][:, None], case, -1.0) for x in g[:2]] + g[2:]
            return torch.cat([x.permute(0, 2, 1, 3) for x in g], 2).flatten(2)
        x = s["qkv"].double().reshape(case["B"], case["T"], -1, d).permute(0, 2, 1, 3)
        turned = _exact_turn(x[:, :hq + hkv], s["pos"][:, None], case)
        return turned[:, :hq], turned[:, hq:], x[:, hq + hkv:]
    x = s["qkv"].double().reshape(-1, hq + 2 * hkv, d)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    if case["bits"] == 16:
        K, V = s["k"].double(), s["v"].double()
    else:
        K, V = _exact_cache(s["k"], s["k_par"], 4), _exact_cache(s["v"], s["v_par"], 8)
    outs = ()
    if case["op"] != "attend":
        q = _exact_turn(q, s["at"][:, None], case)
        k = _exact_turn(k, s["at"][:, None], case)
        if case["bits"] == 4:
            k, v = _exact_hold(k.to(dt)), _exact_hold(v)
        pages, slots = s["table"].long()[s["seq"], s["at"] // case["page"]], s["at"] % case["page"]
        K[pages, :, slots], V[pages, :, slots] = k, v
        outs = (q, K, V) if case["bits"] == 16 else (q, k, v)
        if case["op"] == "append":
            return outs
        q = q.to(dt).double()  # what is attended with is the query in its own type
        if case["bits"] == 16:
            K, V = K.to(dt).double(), V.to(dt).double()
    new = s["at"].shape[0]
    y = torch.empty(new, hq, d, dtype=torch.float64, device=q.device)
    dil = torch.tensor(s["dil"], device=q.device)[:, None]
    for n in range(new):
        p, i = int(s["at"][n]), int(s["seq"][n])
        j = torch.arange(p + 1, device=q.device)
        is_key = ((p - j) % dil == 0) & ((p - j) // dil <= case["r"])
        if s["glob"] is not None:
            is_key |= torch.isin(j, s["glob"][i].long())
        page = s["table"][i].long()[j // case["page"]]
        kk, vv = K[page, :, j % case["page"]].transpose(0, 1), V[page, :, j % case["page"]].transpose(0, 1)
        w = torch.einsum("hgd,hjd->hgj", q[n].reshape(hkv, -1, d), kk) / math.sqrt(d)
        w = torch.softmax(w.masked_fill(~is_key[:, None], -math.inf), -1)
        y[n] = torch.einsum("hgj,hjd->hgd", w, vv).flatten(0, 1)
    return outs + (y,) if outs else y
