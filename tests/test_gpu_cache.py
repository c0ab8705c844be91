"""Rotary positions and the paged cache on the GPU against their definitions in 64 bits (cache_ref), with tolerances
that count the roundings: half a step of the 16-bit type where a value is rounded to it, and a few fp32 steps."""
import math

import pytest
import torch

import oracle
from sparse_long_sequence_fwd_b200 import build, kv_cache, lf_attn, rotary
from tests import cache_ref as ref

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    lf_attn.load()
    lf_attn.device_status()
    yield


@pytest.fixture(autouse=True)
def _no_flags():
    yield
    torch.cuda.synchronize()
    assert lf_attn.device_status() == (0, 0)


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ---------------------------------------------------------------- rotary

def turn_tolerance(x, y, dtype, amplitude):
    """Half a step of the result, and fp32's: angle (2^-24 of half a turn), sine, two products, a sum."""
    size = amplitude * (x.abs() + x.abs().amax(-1, keepdim=True))
    return torch.finfo(dtype).eps / 2 * y.abs() + 2.0 ** -21 * size + (2.0 ** -25 if dtype == F16 else 0.0)


ROTARY = [  # B, T, hq, hkv, d, rot, interleaved, in, out
    (1, 1, 1, 1, 64, 64, False, BF16, BF16),
    (2, 37, 12, 12, 64, 64, False, BF16, BF16),
    (1, 300, 8, 2, 128, 128, True, F16, F16),
    (3, 65, 5, 1, 128, 32, False, F32, F32),
    (2, 129, 4, 4, 64, 24, True, F32, BF16),
    (2, 50, 3, 3, 64, 20, False, BF16, BF16),      # rot that the 16-value items do not divide
    (1, 77, 3, 1, 70, 70, True, F32, F16),         # a head dimension likewise
    (1, 9, 2, 2, 256, 256, False, F16, F16),
    (1, 33, 2, 2, 6, 2, False, F32, F32),
    (2, 20, 4, 4, 64, 0, False, BF16, BF16),       # a copy into another layout
    (1, 700, 3, 1, 80, 80, True, BF16, BF16),      # five items a row
    (2, 311, 1, 1, 48, 16, False, F16, F16),
    (1, 5, 128, 128, 128, 128, False, BF16, BF16),
    (1, 3001, 1, 2, 64, 40, True, BF16, BF16),
]


@pytest.mark.parametrize("case", ROTARY, ids=lambda c: "-".join(str(x) for x in c[:7]))
@pytest.mark.parametrize("inverse", [False, True])
def test_rotary_rows(case, inverse):
    B, T, hq, hkv, d, rot, inter, ti, to = case
    g = gen(T + d)
    packed = torch.randn(B, T, hq + 2 * hkv, d, generator=g).to(ti).cuda()
    q, k, v = (x.transpose(1, 2) for x in packed.split([hq, hkv, hkv], 2))
    f = rotary.freqs(rot, device="cuda")
    pos = torch.randint(0, 1 << 20, (B, T), generator=g, dtype=torch.int32)
    call = rotary.bwd if inverse else rotary.fwd
    got = call(q, k, v, freqs=f, pos=pos.cuda(), interleaved=inter, amplitude=1.25, out_dtype=to)
    for a, x in enumerate((q, k, v)):
        x = x.double().cpu()
        want = x if a == 2 else ref.turn(x, pos[:, None], f.tolist(), inter, 1.25, inverse)
        assert got[a].is_contiguous() and got[a].dtype == to
        off = (got[a].double().cpu() - want).abs()
        assert (off <= turn_tolerance(x, want, to, 1.25)).all(), (a, off.max())


def test_rotary_strides_and_absent_rows():
    g = gen(3)
    f = rotary.freqs(32, scaling="linear", factor=4.0, device="cuda")
    wide = torch.randn(2, 40, 3, 67, generator=g).to(BF16).cuda()
    q = wide[..., 3:67].transpose(1, 2)          # rows off the 16-byte grid
    shared = torch.randn(1, 1, 40, 64, generator=g).to(BF16).cuda().expand(2, 3, 40, 64)  # strides of 0
    out = torch.full((2, 40, 3, 80), 7.0, dtype=BF16, device="cuda")
    where = out[..., 8:72].transpose(1, 2)
    rotary.fwd(None, q, None, freqs=f, out=(None, where, None))
    want = ref.turn(q.double().cpu(), torch.arange(40), f.tolist())
    assert ((where.double().cpu() - want).abs() <= turn_tolerance(q.double().cpu(), want, BF16, 1.0)).all()
    assert (out[..., :8] == 7).all() and (out[..., 72:] == 7).all()
    got = rotary.fwd(shared, freqs=f, pos=torch.full((40,), -5, dtype=torch.int32, device="cuda"))
    want = ref.turn(shared.double().cpu(), torch.full((40,), -5), f.tolist())
    assert got[1] is None and got[2] is None
    assert ((got[0].double().cpu() - want).abs() <= turn_tolerance(shared.double().cpu(), want, BF16, 1.0)).all()
    empty = rotary.fwd(torch.empty(2, 3, 0, 64, dtype=BF16, device="cuda"), freqs=f)
    assert empty[0].shape == (2, 3, 0, 64)


def test_rotary_far_positions_keep_their_angle():
    f = rotary.freqs(64, device="cuda")
    x = torch.randn(1, 1, 4, 64, generator=gen(4)).cuda()
    pos = torch.tensor([2 ** 31 - 1, 2 ** 30 + 1, 16777217, -2 ** 31], dtype=torch.int64)
    got = rotary.fwd(x, freqs=f, pos=pos.to(torch.int32).cuda())[0]
    # the angle, up to 2^31 radians, is formed in fp64 here and there: two roundings each, 2^31 * 2^-53 * 4 radians
    x = x.double().cpu()
    want = ref.turn(x, pos, f.tolist())
    tol = turn_tolerance(x, want, F32, 1.0) + 2.0 ** -20 * x.abs().amax(-1, keepdim=True)
    assert ((got.double().cpu() - want).abs() <= tol).all()


@pytest.mark.parametrize("inter", [False, True])
def test_rotary_gradient_is_that_of_differences(inter):
    """d/dx of sum(g * fwd(x)), by central differences in 64 bits on the definition, against bwd(g)."""
    g = gen(5)
    f = rotary.freqs(12)
    x, up = torch.randn(1, 2, 3, 16, generator=g), torch.randn(1, 2, 3, 16, generator=g)
    got = rotary.bwd(up.cuda(), freqs=f.cuda(), interleaved=inter, amplitude=0.5)[0].double().cpu()
    pos = torch.arange(3)
    loss = lambda z: (ref.turn(z, pos, f.tolist(), inter, 0.5) * up.double()).sum()  # noqa: E731
    for i in range(x.numel()):
        e = torch.zeros(x.numel(), dtype=torch.float64)
        e[i] = 0.5
        e = e.view(x.shape)
        diff = loss(x.double() + e) - loss(x.double() - e)  # the loss is linear: exact but for fp64
        assert abs(diff - got.flatten()[i]) <= 2.0 ** -20 * 4


# ---------------------------------------------------------------- cache

class Step:
    """A step over a cache of random contents: the device tensors, and the CPU copies of what the reference reads."""

    def __init__(self, seed, dtype, bits, new, old, hq, hkv, d, page, r, dil=1, globals_=None, spare_rows=0, pages_more=3):
        g = gen(seed)
        self.dtype, self.bits, self.hq, self.hkv, self.d, self.page, self.r = dtype, bits, hq, hkv, d, page, r
        self.dil = [dil] * hkv if isinstance(dil, int) else dil
        S = len(new)
        per = max(1, max(-(-(a + b) // page) for a, b in zip(new, old)))
        need = [-(-(a + b) // page) for a, b in zip(new, old)]
        pages = sum(need) + pages_more
        self.table = torch.full((S, per), -1, dtype=torch.int32)
        order = torch.randperm(pages, generator=g).to(torch.int32)
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = order[at:at + n]
            at += n
        self.cu = torch.tensor([0] + new).cumsum(0).to(torch.int32)
        self.context = torch.tensor(old, dtype=torch.int32)
        self.N = sum(new) + spare_rows
        self.rows = [(s, old[s] + i) for s in range(S) for i in range(new[s])] + [None] * spare_rows
        self.globals_ = None if globals_ is None else torch.tensor(globals_, dtype=torch.int32)
        if bits == 16:
            self.cpu = [torch.randn(pages, hkv, page, d, generator=g).to(dtype) for _ in range(2)] + [None, None]
        else:
            self.cpu = [torch.randint(0, 256, (pages, hkv, page, d // 2), generator=g, dtype=torch.uint8)
                        for _ in range(2)]
            self.cpu += [torch.stack([0.05 + 0.3 * torch.rand(pages, hkv, page, d // 32, generator=g),
                                      0.3 * torch.randn(pages, hkv, page, d // 32, generator=g)], -1).half()
                         for _ in range(2)]
        self.q = torch.randn(self.N, hq, d, generator=g).to(dtype)
        self.k, self.v = (torch.randn(self.N, hkv, d, generator=g).to(dtype) for _ in range(2))

    def to_gpu(self):
        self.cache = kv_cache.KVCache(*[None if t is None else t.cuda() for t in self.cpu])
        self.plan = kv_cache.Plan(self.cache, self.table.cuda(), self.cu.cuda(), self.context.cuda(), self.N, self.hq,
                                  self.r, dil=self.dil, global_idx=None if self.globals_ is None else self.globals_.cuda())
        return self

    def check(self, got, q=None, scale=None):
        scale = self.d ** -0.5 if scale is None else scale
        q = self.q if q is None else q
        want, by, big = ref.attend(q, self.cpu, self.table, self.rows, self.r, self.dil, self.globals_, scale)
        live = [n for n, at in enumerate(self.rows) if at is not None]
        off = (got.double().cpu() - want)[live].abs()
        tol = ref.attend_tolerance(want, by, big, self.dtype, self.bits)[live]
        assert (off <= tol).all(), ((off / tol).max(), off.max())


FULL = 1 << 30
ATTEND = {  # dtype, bits, new, old, hq, hkv, d, page, r, dil, globals
    "one": (BF16, 16, [1], [0], 1, 1, 64, 8, 0, 1, None),
    "first_tokens": (BF16, 16, [1, 1, 1], [0, 1, 7], 2, 2, 64, 8, 4, 1, None),
    "window": (BF16, 16, [1, 1], [700, 63], 12, 12, 64, 64, 256, 1, [[0], [0]]),
    "window_f16": (F16, 16, [1, 1], [700, 64], 12, 12, 64, 16, 256, 1, [[0], [0]]),
    "dilated": (F16, 16, [1] * 4, [500, 501, 3, 90], 4, 4, 64, 16, 20, [1, 2, 3, 7], [[0, 5, 9, 400]] * 4),
    "duplicates": (BF16, 16, [1, 1], [300, 40], 2, 1, 64, 32, 10, 2, [[9, 3, 3, 290, 9, 296, 295], [500, 0, 39, 40, 0, 7, 7]]),
    "many_globals": (BF16, 16, [1, 1], [900, 130], 2, 2, 64, 64, 30, 1, [list(range(0, 300)), list(range(299, -1, -1))]),
    "shared_5": (BF16, 16, [1, 1], [200, 33], 10, 2, 64, 32, FULL, 1, None),
    "shared_8_d128": (BF16, 16, [1, 1, 1], [1000, 1, 130], 16, 2, 128, 64, FULL, 1, None),
    "shared_12": (F16, 16, [1], [257], 12, 1, 64, 64, 100, 1, [[0, 1]]),
    "shared_16_d128": (BF16, 16, [1], [300], 32, 2, 128, 16, FULL, 1, None),
    "shared_40": (BF16, 16, [2], [300], 40, 1, 64, 16, 64, 1, [[2]]),
    "shared_17": (BF16, 16, [1, 1], [90, 200], 34, 2, 64, 32, 64, 1, [[5, 80]] * 2),
    "shared_20_f16_4": (F16, 4, [1], [300], 20, 1, 64, 32, FULL, 1, None),
    "shared_128": (F16, 16, [1], [65], 128, 1, 128, 256, FULL, 1, None),
    "drafts": (BF16, 16, [5, 0, 3, 1], [100, 10, 0, 63], 4, 2, 64, 32, 16, 1, [[0, 102], [0, 1], [1, 1], [0, 2]]),
    "prompt": (BF16, 16, [150], [0], 2, 1, 64, 64, 32, 1, [[0]]),
    "odd_sequences": (F16, 16, [1] * 17, [13 * i for i in range(17)], 3, 3, 128, 8, 50, 1, None),
    "four": (BF16, 4, [1, 1], [700, 0], 12, 12, 64, 64, 256, 1, [[0], [0]]),
    "four_f16": (F16, 4, [1, 1], [700, 64], 4, 4, 64, 16, 256, 2, [[0, 3], [0, 3]]),
    "four_d128": (BF16, 4, [1, 1], [1100, 31], 8, 2, 128, 32, FULL, 1, None),
    "four_f16_d128_16": (F16, 4, [2], [300], 16, 1, 128, 32, FULL, 1, None),
    "four_shared_12": (BF16, 4, [1], [129], 12, 1, 64, 8, 40, 1, [[0, 64]]),
}


@pytest.mark.parametrize("name", list(ATTEND))
def test_attention_over_the_cache(name):
    s = Step(len(name), *ATTEND[name]).to_gpu()
    s.check(kv_cache.fwd(s.cache, s.plan, s.q.cuda()))
    past = s.globals_ is not None and bool((s.globals_ >= s.table.shape[1] * s.page).any())
    assert lf_attn.device_status() == ((5, 1) if past else (0, 0))  # "duplicates" has a global token behind its table
    if name in ("window", "four_d128"):
        s.check(kv_cache.fwd(s.cache, s.plan, s.q.cuda(), scale=-0.3), scale=-0.3)
        s.check(kv_cache.fwd(s.cache, s.plan, s.q.cuda(), scale=0.0), scale=0.0)


@pytest.mark.parametrize("bits", [16, 4])
def test_long_ragged_batch(bits):
    s = Step(60 + bits, BF16, bits, [1] * 6, [5000, 1, 2047, 64, 63, 900], 6, 3, 64, 64, FULL).to_gpu()
    s.check(kv_cache.fwd(s.cache, s.plan, s.q.cuda()))


def test_more_sequences_and_rows_than_fit_shared_memory():
    """The plan's searches in global memory: 4500 sequences, some without new tokens, and 1500 rows of one."""
    new = [0 if i % 7 == 3 else 1 for i in range(4500)]
    s = Step(70, BF16, 16, new, [i % 13 for i in range(4500)], 2, 1, 64, 8, 6, globals_=[[0, 2]] * 4500).to_gpu()
    s.check(kv_cache.fwd(s.cache, s.plan, s.q.cuda()))
    s = Step(71, F16, 16, [1500, 3], [40, 0], 1, 1, 64, 64, 20, dil=3).to_gpu()
    s.check(kv_cache.fwd(s.cache, s.plan, s.q.cuda()))


def test_a_global_row_sees_every_key():
    s = Step(7, BF16, 16, [1, 3], [1000, 200], 4, 2, 64, 64, 8, dil=[1, 2], globals_=[[0, 1000], [201, 201]]).to_gpu()
    s.check(kv_cache.fwd(s.cache, s.plan, s.q.cuda()))


def test_two_calls_are_equal_bit_for_bit():
    s = Step(8, BF16, 16, [1] * 5, [3000, 20, 777, 64, 1500], 8, 4, 64, 32, FULL).to_gpu()
    q = s.q.cuda()
    a, b = kv_cache.fwd(s.cache, s.plan, q), kv_cache.fwd(s.cache, s.plan, q)
    assert torch.equal(a, b)


@pytest.mark.parametrize("bits", [16, 4])
def test_what_is_no_key_is_never_read(bits):
    """NaN in every slot that is no key of a token: free pages, slots behind the last position, keys outside the window."""
    s = Step(9 + bits, BF16, bits, [1, 1], [100, 37], 4, 2, 64, 32, 10, globals_=[[3], [3]])
    used = torch.zeros(s.cpu[0].shape[:3], dtype=torch.bool)
    for b, p in s.rows:
        for j in ref.key_set(p, 10, 1, s.globals_[b]):
            used[int(s.table[b, j // 32]), :, j % 32] = True
    for t in (s.cpu[:2] if bits == 16 else s.cpu[2:]):
        t[~used] = math.nan
    s.to_gpu()
    got = kv_cache.fwd(s.cache, s.plan, s.q.cuda())
    assert torch.isfinite(got).all()
    s.check(got)


def test_values_of_infinity_and_nan_reach_only_their_rows():
    s = Step(10, BF16, 16, [1, 1], [70, 70], 2, 1, 64, 16, FULL)
    s.cpu[1][int(s.table[0, 1]), 0, 3, 5] = math.inf
    s.cpu[1][int(s.table[0, 2]), 0, 3, 6] = math.nan
    s.to_gpu()
    got = kv_cache.fwd(s.cache, s.plan, s.q.cuda()).double().cpu()
    assert torch.isinf(got[0, :, 5]).all() and torch.isnan(got[0, :, 6]).all()
    fine = [e for e in range(64) if e not in (5, 6)]
    assert torch.isfinite(got[0][:, fine]).all() and torch.isfinite(got[1]).all()


def test_scores_far_apart():
    """Norms that grow along the sequence (the exponent base moves again and again), and keys of score -inf."""
    s = Step(11, BF16, 16, [1], [600], 2, 1, 64, 32, FULL)
    for j in range(601):
        s.cpu[0][int(s.table[0, j // 32]), 0, j % 32] *= 1 + j / 20
    s.to_gpu()
    s.check(kv_cache.fwd(s.cache, s.plan, s.q.cuda()))
    s = Step(12, F16, 16, [1], [100], 2, 1, 64, 32, FULL)
    s.q.abs_()
    for j in range(0, 40):
        s.cpu[0][int(s.table[0, j // 32]), 0, j % 32] = -math.inf  # no part in a row that has other keys
    s.to_gpu()
    s.check(kv_cache.fwd(s.cache, s.plan, s.q.cuda()))


@pytest.mark.parametrize("dtype,bits", [(F16, 16), (BF16, 16), (F16, 4), (BF16, 4)])
def test_a_long_tail_of_small_weights_counts(dtype, bits):
    """One key at score 0 with value 0, and 200000 at about 2^-25.5 of its weight, each under f16's smallest half step,
    with values of 100: their sum is not small."""
    T = 200000
    s = Step(28, dtype, 16, [1], [T - 1], 1, 1, 64, 256, FULL, pages_more=0)
    k, v = torch.zeros(T, 1, 64), torch.zeros(T, 1, 64)
    k[1:, 0, 0], v[1:] = -8.0, 100.0
    s.q.zero_()
    s.q[0, 0, 0] = 17.7
    cu, old = torch.tensor([0, T], dtype=torch.int32).cuda(), torch.zeros(1, dtype=torch.int32).cuda()
    s.bits, s.cache = bits, kv_cache.KVCache.empty(s.cpu[0].shape[0], 1, 256, 64, dtype, bits)
    fill = kv_cache.Plan(s.cache, s.table.cuda(), cu, old, T, 1)
    kv_cache.append(s.cache, fill, k.to(dtype).cuda(), v.to(dtype).cuda())
    s.plan = kv_cache.Plan(s.cache, s.table.cuda(), s.cu.cuda(), s.context.cuda(), 1, 1)
    s.cpu = [None if t is None else t.cpu() for t in (s.cache.k, s.cache.v, s.cache.k_par, s.cache.v_par)]
    got = kv_cache.fwd(s.cache, s.plan, s.q.cuda(), scale=0.125)
    assert 0.2 < got.min() < 1
    s.check(got, scale=0.125)


def test_strides_and_rows_that_are_none():
    s = Step(13, BF16, 16, [2, 1], [40, 9], 6, 2, 64, 16, 20, spare_rows=4).to_gpu()
    packed = torch.randn(s.N, 10, 64, generator=gen(1)).to(BF16)
    packed[:, 2:8] = s.q
    out = torch.full((s.N, 7, 72), 3.0, dtype=BF16, device="cuda")
    got = kv_cache.fwd(s.cache, s.plan, packed.cuda()[:, 2:8], out=out[:, 1:, 5:69])
    s.check(got)
    assert (got[3:] == 3).all() and (out[:, 0] == 3).all() and (out[..., :5] == 3).all() and (out[..., 69:] == 3).all()
    q_out = torch.full_like(s.q.cuda(), 5.0)
    before = s.cache.k.clone()
    kv_cache.append(s.cache, s.plan, s.k.cuda(), s.v.cuda(), q=s.q.cuda(), q_out=q_out)
    assert (q_out[3:] == 5).all() and torch.equal(q_out[:3].cpu(), s.q[:3])
    assert (s.cache.k != before).any(-1).any(1).sum() == 3  # three slots


def test_no_tokens_at_all():
    s = Step(14, BF16, 16, [1], [5], 2, 1, 64, 8, 4)
    s.cu = torch.tensor([0, 0], dtype=torch.int32)
    s.rows = [None]
    s.to_gpu()
    out = torch.full((1, 2, 64), 2.0, dtype=BF16, device="cuda")
    kv_cache.fwd(s.cache, s.plan, s.q.cuda(), out=out)
    assert (out == 2).all()
    s.N = 0
    s.to_gpu()
    assert kv_cache.fwd(s.cache, s.plan, s.q.cuda()[:0]).shape == (0, 2, 64)
    assert kv_cache.append(s.cache, s.plan, s.k.cuda()[:0], s.v.cuda()[:0]) is None


def test_bad_pages_and_positions_are_left_out_and_flagged():
    s = Step(15, BF16, 16, [1, 1, 1], [100, 50, 20], 2, 2, 64, 16, FULL)
    s.table[0, 2], s.table[0, 3] = -1, 1 << 20
    s.table[1, :] = -7                                 # a row without any key: zeros
    s.to_gpu()
    got = kv_cache.fwd(s.cache, s.plan, s.q.cuda())
    s.check(got)
    assert (got[1] == 0).all()
    torch.cuda.synchronize()
    assert lf_attn.device_status() == (5, 4)
    before = s.cache.k.clone()
    s.context[:] = torch.tensor([48, 50, 1 << 20])     # two bad pages, and a position behind the table
    s.to_gpu()
    kv_cache.append(s.cache, s.plan, s.k.cuda(), s.v.cuda())
    out = torch.full((3, 2, 64), 2.0, dtype=BF16, device="cuda")
    kv_cache.fwd(s.cache, s.plan, s.q.cuda(), out=out)
    torch.cuda.synchronize()
    assert torch.equal(s.cache.k, before) and (out[2] == 2).all()
    assert lf_attn.device_status() == (5, 4)
    for bad in ([0, 2, 1, 3], [1, 1, 2, 3], [0, 1, 2, 9]):
        s.cu = torch.tensor(bad, dtype=torch.int32)
        s.to_gpu()
        torch.cuda.synchronize()
        assert lf_attn.device_status()[1] & 4
    s.cu, s.globals_ = torch.tensor([0, 1, 2, 3], dtype=torch.int32), torch.tensor([[0], [-1], [1 << 20]], dtype=torch.int32)
    s.context[:] = 0
    s.to_gpu()
    assert lf_attn.device_status() == (5, 1)


def test_a_plan_of_other_sizes_computes_nothing():
    s = Step(16, BF16, 16, [1, 1], [100, 50], 2, 2, 64, 16, 20).to_gpu()
    out = torch.full((2, 2, 64), 2.0, dtype=BF16, device="cuda")
    s.plan.r = 21
    kv_cache.fwd(s.cache, s.plan, s.q.cuda(), out=out)
    torch.cuda.synchronize()
    assert (out == 2).all() and lf_attn.device_status() == (5, 8)
    before = s.cache.k.clone()
    s.plan.buffer.zero_()
    kv_cache.append(s.cache, s.plan, s.k.cuda(), s.v.cuda())
    assert torch.equal(s.cache.k, before) and lf_attn.device_status() == (5, 8)


# ---------------------------------------------------------------- append

APPEND = [  # dtype, bits, new, old, hq, hkv, d, page, rot, interleaved
    (BF16, 16, [1], [0], 1, 1, 64, 8, 64, False),
    (BF16, 16, [9, 0, 30, 1], [3, 7, 0, 31], 12, 12, 64, 16, 64, False),
    (F16, 16, [70], [100], 8, 2, 128, 64, 32, True),
    (F16, 16, [5, 5], [0, 11], 3, 3, 64, 8, 20, False),
    (BF16, 4, [1], [0], 1, 1, 64, 8, 64, False),
    (BF16, 4, [9, 30, 1], [3, 0, 31], 12, 12, 64, 16, 64, True),
    (F16, 4, [40], [100], 8, 2, 128, 64, 128, False),
    (BF16, 4, [5, 5], [0, 11], 3, 3, 128, 8, 36, True),
    (BF16, 4, [3], [6], 128, 128, 128, 8, 64, False),
]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: "-".join(str(x) for x in c[1:]))
def test_append(case):
    dtype, bits, new, old, hq, hkv, d, page, rot, inter = case
    s = Step(17 + d, dtype, bits, new, old, hq, hkv, d, page, 4, spare_rows=2).to_gpu()
    before = [None if t is None else t.clone() for t in (s.cache.k, s.cache.v, s.cache.k_par, s.cache.v_par)]
    f = rotary.freqs(rot, device="cuda")
    q, hk, hv = kv_cache.append(s.cache, s.plan, s.k.cuda(), s.v.cuda(), q=s.q.cuda(), freqs=f, interleaved=inter,
                                amplitude=1.5, held=True)
    live = torch.tensor([n for n, at in enumerate(s.rows) if at is not None])
    pos = torch.tensor([at[1] for at in s.rows if at is not None])
    page_of = torch.tensor([int(s.table[b, p // page]) for b, p in s.rows[:len(live)]])
    slot = pos % page
    for got, x in ((q, s.q), (hk, s.k)):
        x = x[live].double()
        want = ref.turn(x, pos[:, None], f.tolist(), inter, 1.5)
        if got is q or bits == 16:
            assert ((got.cpu()[live].double() - want).abs() <= turn_tolerance(x, want, dtype, 1.5)).all()
    after = [None if t is None else t.cpu() for t in (s.cache.k, s.cache.v, s.cache.k_par, s.cache.v_par)]
    if bits == 16:
        assert torch.equal(hv.cpu()[live], s.v[live])
        for c, h in ((after[0], hk), (after[1], hv)):
            assert torch.equal(c[page_of, :, slot], h.cpu()[live])
    else:
        codes, par = ref.quantise(s.v[live])  # the values are not turned: codes and parameters are the formula's, exactly
        assert torch.equal(after[1][page_of, :, slot], ref.pack(codes, False))
        assert torch.equal(after[3][page_of, :, slot], par)
        # keys: within half a code of the turned key, or of what rounding it and mid to 16 bits moves
        want = ref.turn(s.k[live].double(), pos[:, None], f.tolist(), inter, 1.5)
        par = after[2][page_of, :, slot]
        have = ref.values(after[0][page_of, :, slot], par, True)[0]
        scale = par[..., :1].double().expand(*par.shape[:-1], 32).flatten(-2)
        assert ((have - want).abs() <= 0.5 * scale + 2.0 ** -7 * want.abs() + 2.0 ** -9 * (want.abs().amax() + 1)).all()
        for c, p, h, is_k in ((0, 2, hk, True), (1, 3, hv, False)):
            x = ref.values(after[c][page_of, :, slot], after[p][page_of, :, slot], is_k)[0]
            assert torch.equal(h.cpu()[live], x.to(dtype))
    for b, a in zip(before, after):  # nothing else has changed
        if b is not None:
            b = b.cpu()
            b[page_of, :, slot] = a[page_of, :, slot]
            assert torch.equal(b.view(torch.uint8), a.view(torch.uint8))


def test_append_into_given_rows_and_without_queries():
    s = Step(19, F16, 4, [6, 2], [250, 9], 4, 2, 64, 256, 4, spare_rows=1).to_gpu()
    wide = torch.full((s.N, 2, 2, 72), 9.0, dtype=F16, device="cuda")
    hk, hv = wide[:, 0, :, 4:68], wide[:, 1, :, 4:68]       # rows off the 16-byte grid
    none, a, b = kv_cache.append(s.cache, s.plan, s.k.cuda(), s.v.cuda(), held=(hk, hv))
    assert none is None and a is hk and b is hv
    for x, h in ((s.k, hk), (s.v, hv)):
        codes, par = ref.quantise(x[:8])
        par = par.double()
        want = (par[..., 1:] + par[..., :1] * (codes.double() - 8).unflatten(-1, (2, 32))).flatten(-2)
        assert torch.equal(h[:8].cpu(), want.to(F16))
    assert (wide[8] == 9).all() and (wide[..., :4] == 9).all() and (wide[..., 68:] == 9).all()


def test_append_quantises_by_the_formula():
    """Untouched keys (no turn): constant groups, single outliers, ties, tiny and large values, infinities and NaN."""
    s = Step(18, BF16, 4, [12], [3], 2, 2, 64, 16, 4)
    k = torch.randn(12, 2, 64, generator=gen(2))
    k[0] = 0
    k[1] = 3.25
    k[2, :, 5] = 1000
    k[3] = torch.arange(64) % 16
    k[4] = (torch.arange(64) % 31) / 2
    k[5] *= 1e-6
    k[6] *= 1e4
    k[7] = -k[7].abs()
    k[8, 0, 3], k[8, 1, 40], k[9, 0, 33] = math.nan, math.inf, -math.inf
    k[10, 0, 3], k[10, 1, 60] = 65536.0, -1e30       # past fp16
    k[11] = 60000 + k[11]
    s.k = k.to(BF16)
    s.to_gpu()
    _, hk, _ = kv_cache.append(s.cache, s.plan, s.k.cuda(), s.v.cuda(), held=True)
    pos = torch.tensor([p for _, p in s.rows])
    page = s.table[0].long()[pos // 16]
    codes, par = ref.quantise(s.k)
    broken = ~(s.k.float().abs() <= 65504).unflatten(-1, (2, 32)).all(-1)
    got_par, got = s.cache.k_par.cpu()[page, :, pos % 16], ref.unpack(s.cache.k.cpu()[page, :, pos % 16], True)
    assert torch.isnan(got_par[..., 1][broken]).all() and torch.isnan(hk.cpu().unflatten(-1, (2, 32))[broken]).all()
    assert torch.equal(got_par[~broken], par[~broken])
    assert torch.equal(got.unflatten(-1, (2, 32))[~broken], codes.unflatten(-1, (2, 32))[~broken])


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("dtype,d,dil", [(BF16, 64, [1, 2]), (F16, 128, [1, 1])])
def test_the_last_row_is_the_forward_passes(dtype, d, dil):
    """A document attended by lf_attn.fwd; its last row again as a token over the cache: the same row."""
    T, H, r, page = 333, 2, 40, 32
    g = gen(20)
    q, k, v = (torch.randn(2, H, T, d, generator=g).to(dtype).cuda() for _ in range(3))
    glob = torch.tensor([[0, 17, 300], [5, T - 1, 5]], dtype=torch.int32).cuda()  # the second document's last row is global
    y = lf_attn.fwd(q, k, v, r, dil=dil, global_idx=glob)
    cache = kv_cache.KVCache.empty(24, H, page, d, dtype)
    table = torch.randperm(24, generator=g)[:22].to(torch.int32).view(2, 11).cuda()
    rows = lambda x, t: x[:, :, t].transpose(1, 2).flatten(0, 1) if isinstance(t, slice) else x[:, :, t]  # noqa: E731
    cu = lambda n: torch.tensor([0, n, 2 * n], dtype=torch.int32).cuda()  # noqa: E731
    old = lambda n: torch.full((2,), n, dtype=torch.int32).cuda()  # noqa: E731
    first = kv_cache.Plan(cache, table, cu(T - 1), old(0), 2 * (T - 1), H, r, dil=dil, global_idx=glob)
    kv_cache.append(cache, first, rows(k, slice(0, T - 1)), rows(v, slice(0, T - 1)))
    step = kv_cache.Plan(cache, table, cu(1), old(T - 1), 2, H, r, dil=dil, global_idx=glob)
    kv_cache.append(cache, step, rows(k, T - 1), rows(v, T - 1))
    got = kv_cache.fwd(cache, step, rows(q, T - 1))
    ref_y = oracle.fwd(q.cpu(), k.cpu(), v.cpu(), r, dil=dil, global_idx=glob.cpu(), scale=d ** -0.5)[:, :, T - 1]
    ref_y = torch.from_numpy(ref_y)
    u = torch.finfo(dtype).eps / 2
    # each of the two rounds P and the output: half a step of values whose weighted sum of magnitudes is under max |v|
    tol = 2 * u * v.abs().max().item() + 1e-5
    assert (got.double().cpu() - ref_y).abs().max() <= tol
    assert (got.double() - y[:, :, T - 1].double()).abs().max() <= 2 * tol


@pytest.mark.parametrize("bits", [16, 4])
def test_prompt_then_tokens(bits):
    """Serving: a prompt appended with its queries turned, then tokens one at a time, each against the definition."""
    hq, hkv, d, page, r = 4, 2, 64, 16, 24
    g = gen(21)
    f = rotary.freqs(48, scaling="ramp", factor=8.0, trained=64, device="cuda")
    cache = kv_cache.KVCache.empty(16, hkv, page, d, BF16, bits)
    table = torch.randperm(16, generator=g).to(torch.int32).view(2, 8)
    glob = torch.tensor([[0, 3], [1, 1]], dtype=torch.int32)
    lens = [0, 0]
    for new in ([37, 50], [1, 1], [1, 1], [2, 0], [1, 1]):
        s = Step(22, BF16, bits, new, lens, hq, hkv, d, page, r, globals_=glob.tolist())
        packed = torch.randn(s.N, hq + 2 * hkv, d, generator=g).to(BF16)
        q, k, v = packed.cuda().split([hq, hkv, hkv], 1)
        s.table = table
        plan = kv_cache.Plan(cache, table.cuda(), s.cu.cuda(), s.context.cuda(), s.N, hq, r, global_idx=glob.cuda())
        qt = kv_cache.append(cache, plan, k, v, q=q, freqs=f, amplitude=1.2, interleaved=True)
        y = kv_cache.fwd(cache, plan, qt)
        s.cpu = [None if t is None else t.cpu() for t in (cache.k, cache.v, cache.k_par, cache.v_par)]
        s.check(y, q=qt.cpu())
        pos = torch.tensor([p for _, p in s.rows])
        want = ref.turn(q.double().cpu(), pos[:, None], f.tolist(), True, 1.2)
        assert ((qt.double().cpu() - want).abs() <= turn_tolerance(q.double().cpu(), want, BF16, 1.2)).all()
        lens = [a + b for a, b in zip(lens, new)]


def test_training_step_through_rotary_and_attention():
    """loss(qkv) = sum(up * attention(turned q, turned k, v)): the gradient of the packed projection that rotary.bwd
    gives behind lf_attn.bwd, against the formula's gradient in 64 bits and against differences."""
    B, T, H, d, r, rot = 1, 40, 2, 16, 5, 12
    g = gen(23)
    packed, up = torch.randn(B, T, 3 * H * d, generator=g), torch.randn(B, H, T, d, generator=g)
    f = rotary.freqs(rot)
    glob = torch.tensor([[0, 11]], dtype=torch.int32)
    split = lambda x: [y.transpose(1, 2) for y in x.unflatten(-1, (3 * H, d)).split([H, H, H], 2)]  # noqa: E731
    gp = packed.cuda()
    q, k, v = rotary.fwd(*split(gp), freqs=f.cuda())
    y = lf_attn.fwd(q, k, v, r, global_idx=glob.cuda())
    grads = lf_attn.bwd(q, k, v, y, up.cuda(), r, global_idx=glob.cuda())
    out = torch.empty_like(gp)
    rotary.bwd(*grads, freqs=f.cuda(), out=split(out))
    got = out.double().cpu()
    mask = torch.tensor([[i in (0, 11) or j in (0, 11) or abs(i - j) <= r for j in range(T)] for i in range(T)])

    def loss(x):
        q, k, v = split(x)
        turned = []
        t = torch.arange(T).double()[:, None] * f
        c, s = t.cos(), t.sin()
        for z in (q, k):
            a, b = z[..., :rot // 2], z[..., rot // 2:rot]
            turned.append(torch.cat([a * c - b * s, b * c + a * s, z[..., rot:]], -1))
        w = (turned[0] @ turned[1].transpose(-1, -2) * d ** -0.5).masked_fill(~mask, -math.inf).softmax(-1)
        return ((w @ v) * up.double()).sum()

    x = packed.double().requires_grad_()
    want, = torch.autograd.grad(loss(x), x)
    # fp32 throughout: sums of up to 40 terms of size max |grad|
    assert (got - want).abs().max() <= 2.0 ** -15 * max(1.0, want.abs().max())
    for i in range(0, packed.numel(), 173):
        e = torch.zeros(packed.numel(), dtype=torch.float64)
        e[i] = 1e-4
        e = e.view(packed.shape)
        diff = (loss(packed.double() + e) - loss(packed.double() - e)) / 2e-4
        assert abs(diff.item() - got.flatten()[i].item()) <= 1e-3 * max(1.0, want.abs().max().item())


# ---------------------------------------------------------------- streams, graphs, size

def test_streams_and_overlapping_calls():
    a = Step(24, BF16, 16, [1] * 3, [900, 30, 400], 4, 2, 64, 32, FULL).to_gpu()
    b = Step(25, F16, 4, [1] * 2, [800, 333], 4, 2, 64, 32, 100).to_gpu()
    qa, qb = a.q.cuda(), b.q.cuda()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    ys = [(kv_cache.fwd(a.cache, a.plan, qa, stream=s1), kv_cache.fwd(b.cache, b.plan, qb, stream=s2)) for _ in range(5)]
    torch.cuda.synchronize()
    for x, y in ys:
        a.check(x)
        b.check(y)
        assert torch.equal(x, ys[0][0]) and torch.equal(y, ys[0][1])


def test_rotary_on_another_stream_than_the_current_one():
    q = torch.randn(2, 3, 5000, 64, generator=gen(6)).cuda()
    f, side = rotary.freqs(64, device="cuda"), torch.cuda.Stream()
    want = rotary.fwd(q, freqs=f)[0]
    x = q.clone()
    torch.cuda.synchronize()
    got = rotary.fwd(x, freqs=f, stream=side)[0]
    del x
    torch.full_like(q, 7.0)  # takes memory of x only once the other stream is done with it
    side.synchronize()
    assert torch.equal(got, want)


def test_captured_step_follows_its_inputs():
    """A captured step (plan, append, attention) replayed with other lengths, queries and page tables; a second
    graph over the same plan between the replays."""
    s = Step(26, BF16, 16, [1, 1], [50, 20], 4, 2, 64, 16, 30, globals_=[[0], [2]], pages_more=6)
    s.table = torch.cat([s.table, torch.full((2, 2), -1, dtype=torch.int32)], 1)
    free = sorted(set(range(s.cpu[0].shape[0])) - set(s.table.flatten().tolist()))
    s.table[0, -2:], s.table[1, -4:] = torch.tensor(free[:2]), torch.tensor(free[2:6])
    s.to_gpu()
    f = rotary.freqs(64, device="cuda")
    q, k, v = s.q.cuda(), s.k.cuda(), s.v.cuda()

    def step():
        s.plan.refresh()
        qt = kv_cache.append(s.cache, s.plan, k, v, q=q, freqs=f)
        return qt, kv_cache.fwd(s.cache, s.plan, qt)

    step()
    torch.cuda.synchronize()
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qt, y = step()
    with torch.cuda.graph(other):
        y2 = kv_cache.fwd(s.cache, s.plan, qt)
    for turn, old in enumerate(([51, 21], [60, 22], [3, 35])):
        g = gen(100 + turn)
        q.copy_(torch.randn(q.shape, generator=g))
        k.copy_(torch.randn(k.shape, generator=g))
        s.plan.context.copy_(torch.tensor(old, dtype=torch.int32))
        graph.replay()
        other.replay()
        torch.cuda.synchronize()
        s.rows = [(0, old[0]), (1, old[1])]
        s.cpu = [s.cache.k.cpu(), s.cache.v.cpu(), None, None]
        s.check(y, q=qt.cpu())
        assert torch.equal(y, y2)
        want = ref.turn(q.double().cpu(), torch.tensor(old)[:, None], f.tolist())
        assert ((qt.double().cpu() - want).abs() <= turn_tolerance(q.double().cpu(), want, BF16, 1.0)).all()


def test_cache_past_32_bit_offsets():
    """Pages behind 2^32 bytes: the last page of caches of 4.4 GB."""
    pages, hkv, page, d = 4200, 16, 256, 128
    cache = kv_cache.KVCache.empty(pages, hkv, page, d, BF16)
    s = Step(27, BF16, 16, [1], [300], hkv, hkv, d, page, FULL, pages_more=0)
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32)
    for i in range(2):
        for c, cpu in ((cache.k, s.cpu[0]), (cache.v, s.cpu[1])):
            c[pages - 1 - i] = cpu[int(s.table[0, i])].cuda()
    plan = kv_cache.Plan(cache, table.cuda(), s.cu.cuda(), s.context.cuda(), 1, hkv, FULL)
    s.check(kv_cache.fwd(cache, plan, s.q.cuda()))
    kv_cache.append(cache, plan, s.k.cuda(), s.v.cuda())
    assert torch.equal(cache.k[pages - 2, :, 300 - 256].cpu(), s.k[0])


PACKED = {  # rows of a sequence that are taken together: dtype, bits, new, old, hq, hkv, d, page, r, dil, globals
    "two_each": (BF16, 16, [2] * 100, list(range(0, 300, 3)), 4, 4, 64, 16, 30, 1, None),
    "drafts": (F16, 16, [4, 7, 0, 5] * 12, list(range(300, 348)), 8, 4, 64, 64, 256, 1, [[0, 302, 310]] * 48),
    "prompt": (BF16, 16, [333], [0], 3, 3, 64, 64, 100, 1, [[0, 40, 41, 200, 332]]),
    "prompt_behind_one": (F16, 16, [320, 1], [70, 2000], 6, 2, 64, 8, 64, 1, [[0, 64, 65, 69], [0, 1, 2, 1999]]),
    "window_0": (BF16, 16, [500, 120], [17, 0], 1, 1, 64, 16, 0, 1, [[3, 17, 30], [0, 119, 5]]),
    "window_1": (F16, 16, [640, 3], [0, 0], 1, 1, 64, 32, 1, 1, None),
    "many_globals": (BF16, 16, [400, 300], [0, 500], 2, 1, 64, 64, 7, 1, [list(range(0, 400, 2)), list(range(500, 100, -2))]),
    "shared_3": (BF16, 16, [300, 19], [9, 3], 6, 2, 64, 32, FULL, 1, None),
    "shared_5_d128": (F16, 16, [200], [130], 10, 2, 128, 64, 60, 1, [[0, 5]]),
    "shared_4_d128": (BF16, 16, [160, 2], [70, 40], 8, 2, 128, 16, FULL, 1, None),
    "long": (BF16, 16, [8, 3], [5000, 64], 4, 1, 64, 256, FULL, 1, None),
    "wide_window": (F16, 16, [4, 2, 4], [3000, 50, 1300], 8, 8, 128, 32, 900, 1, None),
    "no_tile": (BF16, 16, [600], [100], 2, 2, 64, 16, 20, 2, [[0]]),          # dilated: row by row
    "four": (BF16, 4, [150, 2], [0, 500], 4, 4, 64, 64, 50, 1, [[0, 30], [0, 3]]),
    "four_f16": (F16, 4, [5, 3, 9], [100, 1000, 3], 8, 2, 64, 16, FULL, 1, None),
    "four_d128": (BF16, 4, [4, 4], [3000, 31], 8, 8, 128, 32, FULL, 1, None),
    "four_f16_d128": (F16, 4, [200], [128], 12, 3, 128, 64, 90, 1, [[0, 128, 164]]),
}


@pytest.mark.parametrize("name", list(PACKED))
def test_rows_taken_together(name):
    s = Step(100 + len(name), *PACKED[name]).to_gpu()
    q = s.q.cuda()
    got = kv_cache.fwd(s.cache, s.plan, q)
    s.check(got)
    s.check(kv_cache.fwd(s.cache, s.plan, q, scale=-0.2), scale=-0.2)
    assert torch.equal(got, kv_cache.fwd(s.cache, s.plan, q))


@pytest.mark.parametrize("dtype,bits,d,hq", [(BF16, 16, 64, 4), (F16, 16, 128, 2), (BF16, 4, 128, 2), (F16, 4, 64, 6)])
def test_a_row_of_a_tile_does_not_meet_its_neighbours_keys(dtype, bits, d, hq):
    """No number, in K or in V, at keys that some rows of a tile see: those rows have none, the others are finite and as
    without it.  Among them list entries: one that rows from 200 on see, one that a whole sequence sees."""
    for bad in (math.nan, math.inf):
        for which in (0, 1):
            s = Step(200, dtype, bits, [300, 5], [0, 50], hq, 2, d, 16, 10, globals_=[[200, 31], [3, 3]], pages_more=0)
            clean = [None if t is None else t.clone() for t in s.cpu]
            hit = {(0, j) for j in range(28, 200, 37)} | {(1, 52)} | ({(0, 200), (1, 3)} if which else set())
            for b, j in hit:
                at = int(s.table[b, j // 16]), slice(None), j % 16
                if bits == 16:
                    s.cpu[which][at] = bad
                else:
                    s.cpu[2 + which][at][..., 1] = bad
            s.to_gpu()
            got = kv_cache.fwd(s.cache, s.plan, s.q.cuda()).double().cpu()
            s.cpu = clean
            want, by, big = ref.attend(s.q, s.cpu, s.table, s.rows, s.r, s.dil, s.globals_, d ** -0.5)
            tol = ref.attend_tolerance(want, by, big, dtype, bits)
            for n, (b, p) in enumerate(s.rows):
                keys = set(ref.key_set(p, 10, 1, s.globals_[b]))
                if any((b, j) in hit for j in keys):
                    if which or bad != bad:
                        assert not torch.isfinite(got[n]).any(), (n, b, p)
                else:
                    assert ((got[n] - want[n]).abs() <= tol[n]).all(), (n, b, p)


def test_infinite_values_without_weight_in_a_tile():
    """A value of infinity whose weight is 0 in 64 bits too (scores 80 and -8000: e^-8080): no number in every row that
    sees it, as 0 times infinity is none, and nothing in the others."""
    s = Step(201, BF16, 16, [620], [30], 1, 1, 64, 16, 12)
    s.q.zero_()
    s.q[:, 0, 0] = 8.0
    at = int(s.table[0, 2]), 0, 3  # position 35
    s.cpu[0][:, :, :, 0] = 10.0
    s.cpu[0][at][0] = -1000.0
    s.cpu[1][at][5] = math.inf
    s.to_gpu()
    got = kv_cache.fwd(s.cache, s.plan, s.q.cuda(), scale=1.0).double().cpu()
    for n, (_, p) in enumerate(s.rows):
        assert not torch.isfinite(got[n, 0, 5]) if p - 12 <= 35 <= p else torch.isfinite(got[n]).all(), p
        assert torch.isfinite(got[n, 0, 6])


def test_rows_taken_together_and_bad_pages_tables_and_strides():
    """Pages outside the cache hold no keys, rows behind the table are none, rows behind the last sequence stay; queries
    and outputs are rows of wider tensors."""
    s = Step(202, F16, 16, [280, 21], [40, 10], 4, 2, 64, 16, 25, globals_=[[0, 33], [1, 2]], spare_rows=7)
    s.table[0, 2], s.table[1, 0] = -5, 1 << 20
    s.to_gpu()
    wide = torch.zeros(s.N, 5, 3, 64, dtype=F16, device="cuda")
    q = wide[:, 1:5, 1]
    q.copy_(s.q)
    out = torch.full((s.N, 4, 2, 64), 7.0, dtype=F16, device="cuda")
    got = kv_cache.fwd(s.cache, s.plan, q, out=out[:, :, 1])
    assert lf_attn.device_status()[0] & 4
    s.check(got)
    assert (out[:, :, 0] == 7).all() and (out[301:] == 7).all()

    s = Step(203, BF16, 16, [304], [40], 2, 2, 64, 16, 25)
    s.context += 16  # the last 8 rows are behind the table
    s.rows = [(0, 56 + i) if i < 296 else None for i in range(304)]
    s.to_gpu()
    out = torch.full((304, 2, 64), 7.0, dtype=BF16, device="cuda")
    s.check(kv_cache.fwd(s.cache, s.plan, s.q.cuda(), out=out))
    assert lf_attn.device_status()[0] & 4
    assert (out[296:] == 7).all()


def test_prompt_and_drafts_in_a_captured_step():
    """A captured step whose sequences take other rows on replay: tiles are made anew."""
    s = Step(204, BF16, 16, [200, 120], [100, 200], 4, 2, 64, 32, 50, globals_=[[0, 110], [0, 7]]).to_gpu()
    q, cu, old = s.q.cuda(), s.cu.cuda(), s.context.cuda()
    table, listed = s.table.cuda(), s.globals_.cuda()

    def step():
        plan = kv_cache.Plan(s.cache, table, cu, old, s.N, 4, 50, global_idx=listed)
        return kv_cache.fwd(s.cache, plan, q)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for new, before in (([200, 120], [100, 200]), ([1, 300], [119, 20]), ([290, 0], [10, 5])):
        cu.copy_(torch.tensor([0, new[0], sum(new)], dtype=torch.int32))
        old.copy_(torch.tensor(before, dtype=torch.int32))
        s.rows = [(b, before[b] + i) for b in range(2) for i in range(new[b])]
        graph.replay()
        torch.cuda.synchronize()
        s.check(got)


# ---------------------------------------------------------------- rows that 16-value items do not divide

PARTS = [  # rotary: B, T, hq, hkv, d, rot, interleaved, in, out
    (1, 40, 3, 2, 64, 2, False, BF16, BF16),
    (2, 301, 12, 4, 64, 24, False, BF16, BF16),    # two pairs at a time
    (1, 77, 5, 5, 64, 62, False, F16, F16),        # one
    (1, 33, 9, 1, 128, 100, False, F32, BF16),
    (3, 19, 17, 1, 128, 90, False, F32, F32),
    (2, 50, 40, 8, 128, 60, True, BF16, BF16),     # rot ends inside a chunk
    (1, 64, 2, 2, 64, 2, True, F32, F16),
    (1, 21, 3, 3, 96, 70, True, BF16, BF16),
    (1, 700, 2, 1, 256, 252, False, F16, F16),
    (1, 5, 2, 1, 255, 254, False, F32, F32),       # 127 pairs and one value
    (2, 9, 1, 1, 1, 0, False, BF16, BF16),
]


@pytest.mark.parametrize("case", PARTS, ids=lambda c: "-".join(str(x) for x in c[:7]))
@pytest.mark.parametrize("inverse", [False, True])
def test_rotary_rows_by_pairs(case, inverse):
    test_rotary_rows(case, inverse)


@pytest.mark.parametrize("case", [  # dtype, bits, new, old, hq, hkv, d, page, rot, interleaved
    (BF16, 16, [40, 3], [0, 9], 12, 4, 64, 16, 24, False),
    (F16, 16, [1, 9], [60, 0], 6, 2, 64, 8, 62, False),
    (F16, 16, [130], [7], 2, 2, 128, 64, 52, True),
    (BF16, 4, [33, 2], [0, 77], 4, 4, 64, 32, 24, False),
    (F16, 4, [17], [20], 8, 1, 128, 16, 90, False),
    (BF16, 4, [5, 600], [20, 0], 5, 5, 128, 16, 100, False),
    (F16, 4, [6], [0], 3, 3, 64, 8, 2, True),
], ids=lambda c: "-".join(str(x) for x in c[1:]))
def test_append_by_pairs(case):
    test_append(case)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot", [2, 12, 22, 36, 60])
def test_values_behind_rot_are_copies(inter, rot):
    """Infinities and NaN behind rot stay what they are and where they are."""
    g = gen(300 + rot)
    x = torch.randn(1, 3, 50, 64, generator=g)
    x[..., rot:] = torch.tensor([math.inf, -math.inf, math.nan, 1.5])[torch.randint(0, 4, (1, 3, 50, 64 - rot), generator=g)]
    x = x.to(BF16).cuda()
    got = rotary.fwd(x, freqs=rotary.freqs(rot, device="cuda"), interleaved=inter)[0]
    assert torch.isfinite(got[..., :rot]).all()
    assert torch.equal(got[..., rot:].nan_to_num(9.0), x[..., rot:].nan_to_num(9.0))


@pytest.mark.parametrize("shift", [0, 1, 2, 4])
@pytest.mark.parametrize("bits", [16, 4])
def test_outputs_at_any_place(bits, shift):
    """Outputs whose rows begin on 2, 4 and 8 bytes, of whole units and of cut ones, single rows and tiles."""
    for seed, new, old, r in ((400, [1, 1], [700, 5], 100), (401, [1], [3000], FULL), (402, [400], [9], 40)):
        s = Step(seed, F16, bits, new, old, 4, 2, 128, 32, r).to_gpu()
        out = torch.full((s.N, 4, 132 + shift % 4), 3.0, dtype=F16, device="cuda")
        got = kv_cache.fwd(s.cache, s.plan, s.q.cuda(), out=out[..., shift:shift + 128])
        s.check(got)
        assert (out[..., :shift] == 3).all() and (out[..., shift + 128:] == 3).all()
