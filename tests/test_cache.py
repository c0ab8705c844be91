"""What the rotary positions and the paged cache refuse, before anything touches a GPU, and the frequencies."""
import ctypes
import math

import pytest
import torch

from sparse_long_sequence_fwd_b200 import build, kv_cache, lf_attn, rotary
from tests import cache_ref as ref


@pytest.fixture(scope="module")
def lib():
    build.build()
    return lf_attn.load()


P = ctypes.c_void_p
FAKE = 1 << 20
OK, INVALID, UNSUPPORTED, SMALL = 0, 1, 2, 6


def i64(*x):
    return (ctypes.c_int64 * len(x))(*x)


def i32(*x):
    return (ctypes.c_int32 * len(x))(*x)


def call(fn, args, order, **kw):
    a = dict(args, **kw)
    return fn(*[P(a[n]) if isinstance(a[n], int) and n in a["_p"] else a[n] for n in order])


ROTARY = dict(q=FAKE, k=2 * FAKE, v=3 * FAKE, qo=4 * FAKE, ko=5 * FAKE, vo=6 * FAKE,
              s=i64(*[8192, 4096, 64] * 6), B=2, hq=2, hkv=2, T=64, d=64, pos=None, ps=0, f=7 * FAKE, rot=64, inter=0,
              inv=0, amp=1.0, ti=1, to=1, stream=None, _p=("q", "k", "v", "qo", "ko", "vo", "f", "pos"))
ROTARY_ORDER = ("q k v qo ko vo s B hq hkv T d pos ps f rot inter inv amp ti to stream").split()


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), INVALID), (dict(q=None, qo=None, k=None, ko=None, v=None, vo=None), INVALID), (dict(s=None), INVALID),
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(d=0), INVALID), (dict(hq=-1), INVALID),
    (dict(rot=63), INVALID), (dict(rot=66), INVALID), (dict(rot=-2), INVALID), (dict(f=None), INVALID),
    (dict(amp=math.inf), INVALID), (dict(ti=3), INVALID), (dict(to=-1), INVALID), (dict(ps=-1), INVALID),
    (dict(q=FAKE + 1), INVALID), (dict(f=FAKE + 4), INVALID), (dict(pos=FAKE + 2), INVALID),
    (dict(qo=FAKE), INVALID), (dict(qo=2 * FAKE + 100), INVALID),                # outputs over inputs
    (dict(s=i64(*[8192, 4096, 64] * 3 + [0, 4096, 64] * 3)), INVALID),           # rows written over one another
    (dict(s=i64(*[-8192, 4096, 64] * 6)), INVALID), (dict(s=i64(*[1 << 60, 4096, 64] * 6)), INVALID),
    (dict(ti=1, to=0), UNSUPPORTED), (dict(ti=1, to=2), UNSUPPORTED), (dict(d=258), UNSUPPORTED),
    (dict(B=65536, s=i64(*[1, 1, 1] * 6), q=FAKE, qo=1 << 30, k=None, ko=None, v=None, vo=None), UNSUPPORTED),
    (dict(s=i64(*[0, 1 << 31, 64] + [8192, 4096, 64] * 5), T=2), UNSUPPORTED),
    (dict(B=0), OK), (dict(T=0), OK), (dict(hq=0, hkv=0), OK),
])
def test_rotary_refusals(lib, kw, code):
    assert call(lib.lf_attn_rotary, ROTARY, ROTARY_ORDER, **kw) == code


PLAN = dict(cu=FAKE, ctx=FAKE, S=2, N=2, g=None, ng=0, page=16, mp=8, hq=4, hkv=2, d=64, bits=16, r=5, dil=None, plan=FAKE, stream=None,
            _p=("cu", "ctx", "g", "plan"))
PLAN_ORDER = "cu ctx S N g ng page mp hq hkv d bits r dil plan stream".split()


@pytest.mark.parametrize("kw,code", [
    (dict(cu=None), INVALID), (dict(ctx=None), INVALID), (dict(plan=None), INVALID), (dict(plan=FAKE + 128), INVALID),
    (dict(ng=2), INVALID), (dict(g=FAKE), INVALID), (dict(ng=-1), INVALID), (dict(S=0), INVALID), (dict(N=-1), INVALID),
    (dict(page=0), INVALID), (dict(mp=0), INVALID), (dict(hq=3), INVALID), (dict(hkv=0), INVALID), (dict(r=-1), INVALID),
    (dict(dil=i32(1, 0)), INVALID), (dict(cu=FAKE + 2), INVALID), (dict(bits=8), INVALID), (dict(d=0), INVALID),
    (dict(d=96), UNSUPPORTED),
    (dict(page=4), UNSUPPORTED), (dict(page=48), UNSUPPORTED), (dict(page=512), UNSUPPORTED), (dict(hq=256), UNSUPPORTED),
    (dict(g=FAKE, ng=1025), UNSUPPORTED), (dict(mp=1 << 27), UNSUPPORTED), (dict(N=(1 << 20) + 1), UNSUPPORTED),
    (dict(S=(1 << 20) + 1), UNSUPPORTED),
])
def test_plan_refusals(lib, kw, code):
    assert call(lib.lf_attn_cache_plan, PLAN, PLAN_ORDER, **kw) == code


def test_sizes(lib):
    assert lib.lf_attn_cache_plan_bytes(1, 0, 0) > 0
    for bad in ((0, 1, 0), (1, -1, 0), (1, 1, -1), (1, 1, 1025), ((1 << 20) + 1, 1, 0)):
        assert lib.lf_attn_cache_plan_bytes(*bad) == 0
    size = lambda n=1, ng=0, page=16, mp=1000, hq=12, hkv=12, d=64, bits=16, r=1 << 30: (  # noqa: E731
        lib.lf_attn_cache_workspace_bytes(n, ng, page, mp, hq, hkv, d, bits, r))
    assert size() > 0 and size(hq=24) > size() and size(r=5000) > 0
    assert size(r=100) == 0 and size(mp=2) == 0        # windows, or tables, that no CTA needs help with
    assert size(n=10000, r=1000) == 0                  # or rows enough for all
    for bad in (dict(hkv=5), dict(hq=0), dict(d=96), dict(hq=256, hkv=1), dict(bits=8), dict(ng=-1), dict(n=-1)):
        assert size(**bad) == 0


APPEND = dict(k=FAKE, v=2 * FAKE, q=3 * FAKE, hk=None, hv=None, qo=4 * FAKE, s=i64(*[256, 64] * 6), kc=5 * FAKE, vc=6 * FAKE,
              kp=None, vp=None, pages=8, page=16, table=FAKE, mp=8, plan=FAKE, S=2, N=2, ng=0, hq=4, hkv=2, d=64, f=FAKE,
              rot=64, inter=0, amp=1.0, t=1, bits=16, stream=None,
              _p=("k", "v", "q", "hk", "hv", "qo", "kc", "vc", "kp", "vp", "table", "plan", "f"))
APPEND_ORDER = "k v q hk hv qo s kc vc kp vp pages page table mp plan S N ng hq hkv d f rot inter amp t bits stream".split()


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(q=None), INVALID), (dict(qo=None), INVALID),
    (dict(table=None), INVALID), (dict(plan=None), INVALID), (dict(kc=None), INVALID), (dict(kc=FAKE + 8), INVALID),
    (dict(kp=FAKE, vp=FAKE), INVALID), (dict(bits=4), INVALID), (dict(bits=4, kp=FAKE), INVALID), (dict(bits=8), INVALID),
    (dict(rot=66), INVALID), (dict(rot=1), INVALID), (dict(f=None), INVALID), (dict(amp=math.nan), INVALID),
    (dict(pages=0), INVALID), (dict(k=FAKE + 1), INVALID), (dict(qo=3 * FAKE + 64), INVALID), (dict(hk=FAKE), INVALID),
    (dict(s=i64(*[256, 64] * 5 + [256, 0])), INVALID), (dict(t=5), INVALID),
    (dict(t=0), UNSUPPORTED), (dict(d=32, rot=32), UNSUPPORTED), (dict(pages=1 << 27), UNSUPPORTED),
    (dict(page=24), UNSUPPORTED), (dict(s=i64(*[1 << 31, 64] + [256, 64] * 5), k=1 << 40), UNSUPPORTED), (dict(N=0), OK),
])
def test_append_refusals(lib, kw, code):
    assert call(lib.lf_attn_cache_append, APPEND, APPEND_ORDER, **kw) == code


FWD = dict(q=FAKE, o=2 * FAKE, s=i64(256, 64, 256, 64), kc=3 * FAKE, vc=3 * FAKE, kp=None, vp=None, pages=8, page=16,
           table=FAKE, mp=8, plan=FAKE, S=2, N=2, ng=0, hq=4, hkv=2, d=64, r=5, dil=None, scale=0.125, t=1, bits=16,
           ws=FAKE, wb=1 << 30, stream=None, _p=("q", "o", "kc", "vc", "kp", "vp", "table", "plan", "ws"))
FWD_ORDER = "q o s kc vc kp vp pages page table mp plan S N ng hq hkv d r dil scale t bits ws wb stream".split()


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), INVALID), (dict(o=None), INVALID), (dict(ws=None, r=5000, mp=1000), INVALID), (dict(ws=FAKE + 8), INVALID), (dict(plan=None), INVALID),
    (dict(table=None), INVALID), (dict(scale=math.nan), INVALID), (dict(q=FAKE + 2), INVALID), (dict(o=2 * FAKE + 1), INVALID),
    (dict(o=FAKE + 128), INVALID), (dict(s=i64(260, 64, 256, 64)), INVALID), (dict(s=i64(256, 64, 0, 64)), INVALID),
    (dict(s=i64(256, -64, 256, 64)), INVALID), (dict(r=-1), INVALID), (dict(dil=i32(0, 1)), INVALID),
    (dict(bits=4), INVALID), (dict(t=0), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(wb=1000, r=5000, mp=1000), SMALL), (dict(N=0), OK),
])
def test_attention_refusals(lib, kw, code):
    assert call(lib.lf_attn_cache_fwd, FWD, FWD_ORDER, **kw) == code


def test_binding_refusals():
    x = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    f = rotary.freqs(64)
    for kw, err in ((dict(q=x, freqs=f), ValueError),                                     # no CUDA tensor
                    (dict(q=None, freqs=f), ValueError), (dict(q=x[0], freqs=f), ValueError),
                    (dict(q=x, k=x[:, :, :3], freqs=f), ValueError), (dict(q=x, k=x.half(), freqs=f), TypeError),
                    (dict(q=x, freqs=f.float()), ValueError), (dict(q=x[..., :32], freqs=f), ValueError),
                    (dict(q=x, freqs=f, pos=torch.arange(4)), ValueError),
                    (dict(q=x, freqs=f, pos=torch.zeros(3, dtype=torch.int32)), ValueError),
                    (dict(q=x, freqs=f, out=(x,)), ValueError), (dict(q=x, freqs=f, out=(None, x, None)), ValueError),
                    (dict(q=x.transpose(2, 3), freqs=rotary.freqs(4)), ValueError),
                    (dict(q=x.to(torch.float64), freqs=f), TypeError)):
        with pytest.raises(err):
            rotary.fwd(**kw)
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    u = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    h = lambda *s: torch.zeros(*s, dtype=torch.float16)  # noqa: E731
    for args, err in (((z(2, 1, 8, 64), z(2, 1, 8, 32)), ValueError), ((z(2, 1, 8), z(2, 1, 8)), ValueError),
                      ((u(2, 1, 8, 32), u(2, 1, 8, 32)), TypeError),
                      ((u(2, 1, 8, 32), u(2, 1, 8, 32), h(2, 1, 8, 2, 2)), ValueError),
                      ((u(2, 1, 8, 32), u(2, 1, 8, 32), h(2, 1, 8, 1, 2), h(2, 1, 8, 1, 2)), ValueError),
                      ((z(2, 1, 8, 32), z(2, 1, 8, 32), h(2, 1, 8, 2, 2), h(2, 1, 8, 2, 2)), TypeError),
                      ((z(2, 8, 1, 64).transpose(1, 2), z(2, 8, 1, 64).transpose(1, 2).contiguous()), ValueError)):
        if args[0].is_contiguous() and err is ValueError and args[0].shape == (2, 1, 8, 64) and len(args) == 2 and \
                args[1].shape == args[0].shape:
            continue
        with pytest.raises(err):
            kv_cache.KVCache(*args)
    cache = kv_cache.KVCache(z(4, 2, 8, 64), z(4, 2, 8, 64))
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    for args in ((i(2, 3), i(2), i(2), 2, 4), (i(3, 3), i(3), i(2), 2, 4), (i(2, 3).long(), i(3), i(2), 2, 4),
                 (i(2, 3), i(3), i(2, 1), 2, 4), (i(2, 3), i(3), i(2), 2, 4)):              # the last: not on a GPU
        with pytest.raises(ValueError):
            kv_cache.Plan(cache, *args, r=3)


def test_frequencies():
    f = rotary.freqs(8)
    assert f.dtype == torch.float64
    assert torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64), rtol=1e-15)
    assert torch.equal(rotary.freqs(8, scaling="linear", factor=4.0), f / 4)
    based = rotary.freqs(8, scaling="base", factor=4.0)
    assert based[0] == 1 and math.isclose(based[-1], f[-1] / 4, rel_tol=1e-12)
    ramp = rotary.freqs(8, scaling="ramp", factor=4.0, trained=1000, turns=(1.0, 32.0))
    # turns in 1000 positions: 159, 15.9, 1.59, 0.159: kept, blended, blended, divided
    assert ramp[0] == f[0] and ramp[3] == f[3] / 4
    keep = (100 / (2 * math.pi) - 1) / 31
    assert math.isclose(ramp[1], 0.1 * keep + 0.025 * (1 - keep), rel_tol=1e-12)
    assert rotary.freqs(0).numel() == 0
    for kw in (dict(rot=3), dict(rot=-2), dict(rot=8, scaling="other"), dict(rot=8, scaling="ramp"), dict(rot=2, scaling="base"),
               dict(rot=8, factor=0.0), dict(rot=8, scaling="ramp", trained=10, turns=(3.0, 1.0))):
        with pytest.raises(ValueError):
            rotary.freqs(**kw)


def test_the_packing_is_one_to_one():
    for d in (64, 128):
        for is_k in (True, False):
            c = torch.randint(0, 16, (5, d), generator=torch.Generator().manual_seed(d))
            assert sorted(ref.place(d, is_k).tolist()) == list(range(d))
            assert torch.equal(ref.unpack(ref.pack(c, is_k), is_k), c)


def test_strided_cache_tensors_are_refused():
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    u = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    h = lambda *s: torch.zeros(*s, dtype=torch.float16)  # noqa: E731
    bad = z(2, 8, 2, 64).transpose(1, 2)
    assert not bad.is_contiguous()
    for args in ((bad, z(2, 2, 8, 64)), (z(2, 2, 8, 64), bad), (z(2, 2, 8, 128)[..., :64], z(2, 2, 8, 64)),
                 (u(2, 2, 8, 32), u(2, 2, 8, 64)[..., ::2], h(2, 2, 8, 2, 2), h(2, 2, 8, 2, 2)),
                 (u(2, 2, 8, 32), u(2, 2, 8, 32), h(2, 2, 8, 2, 2), h(2, 2, 2, 8, 2).transpose(2, 3))):
        with pytest.raises(ValueError, match="contiguous"):
            kv_cache.KVCache(*args)


def test_sizes_past_32_bits_do_not_wrap():
    cache = kv_cache.KVCache(torch.zeros(4, 2, 8, 64).half(), torch.zeros(4, 2, 8, 64).half())
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    for kw in (dict(r=-1), dict(r=-(1 << 32) + 5), dict(r=3, dil=0), dict(r=3, dil=[1, 1 - (1 << 32)])):
        with pytest.raises(ValueError, match="r must|dil must"):
            kv_cache.Plan(cache, i(2, 3), i(3), i(2), 2, 4, **kw)
    for kw in (dict(n_tokens=(1 << 32) + 2, q_heads=4), dict(n_tokens=2, q_heads=(1 << 32) + 4), dict(n_tokens=-1, q_heads=4),
               dict(n_tokens=2, q_heads=0)):
        with pytest.raises(ValueError, match="n_tokens|q_heads"):
            kv_cache.Plan(cache, i(2, 3), i(3), i(2), r=3, **kw)


@pytest.mark.parametrize("what,kw", [
    ("rotary", dict(ko=4 * FAKE)), ("rotary", dict(qo=6 * FAKE)),                     # two outputs in one place
    ("rotary", dict(s=i64(*[8192, 4096, 64] * 5 + [8192, 4096, 63]))),                # rows that reach into the next
    ("rotary", dict(s=i64(*[8192, 4096, 64] * 3 + [8192, 64, 64] + [8192, 4096, 64] * 2))),      # heads on tokens
    ("rotary", dict(s=i64(*[8192, 4096, 64] * 4 + [4032, 4096, 64] + [8192, 4096, 64]))),         # samples on heads
    ("append", dict(hk=7 * FAKE, hv=7 * FAKE)), ("append", dict(hk=4 * FAKE)), ("append", dict(vc=5 * FAKE)),
    ("append", dict(hv=5 * FAKE)), ("append", dict(s=i64(*[256, 64] * 5 + [128, 64]))),
    ("append", dict(bits=4, kp=8 * FAKE, vp=8 * FAKE)),
    ("fwd", dict(s=i64(256, 64, 256, 32))), ("fwd", dict(s=i64(256, 64, 192, 64))), ("fwd", dict(s=i64(256, 64, 64, 64))),
])
def test_outputs_that_lie_on_one_another_are_refused(lib, what, kw):
    fn, args, order = {"rotary": (lib.lf_attn_rotary, ROTARY, ROTARY_ORDER), "fwd": (lib.lf_attn_cache_fwd, FWD, FWD_ORDER),
                       "append": (lib.lf_attn_cache_append, APPEND, APPEND_ORDER)}[what]
    assert call(fn, args, order, **kw) == INVALID
