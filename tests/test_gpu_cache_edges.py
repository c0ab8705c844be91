"""The paged cache at the ends of its types and shapes, against the definitions in 64 bits."""
import math

import pytest
import torch

from sparse_long_sequence_fwd_b200 import kv_cache, lf_attn, rotary
from tests import cache_ref as ref
from tests.test_gpu_cache import BF16, F16, FULL, Step, _lib, _no_flags, gen, turn_tolerance  # noqa: F401

pytestmark = pytest.mark.gpu


FORMS = {  # new, old, hq, hkv, r: single rows of one and of two tiles of heads, cut ones, tiles of rows
    "single": ([1, 1], [300, 45], 4, 2, 100),
    "heads_12": ([1], [400], 12, 1, 200),
    "cut": ([1], [1500], 4, 2, FULL),
    "tiles": ([330, 5], [40, 70], 4, 2, 70),
    "tiles_of_one_head": ([650], [60], 1, 1, 120),
}


@pytest.mark.parametrize("dtype,d", [(F16, 64), (BF16, 64), (F16, 128), (BF16, 128)])
@pytest.mark.parametrize("form", list(FORMS))
def test_4_bit_values_past_the_largest_fp16(form, dtype, d):
    """Groups from -65504 to 65504 (scale 8736, mid 4384) and near one end, whose outer codes stand for 65536 and -65536, and
    one that no append makes, down to -74272."""
    new, old, hq, hkv, r = FORMS[form]
    s = Step(500 + d, dtype, 4, new, old, hq, hkv, d, 16, r)
    par = torch.tensor([[8736.0, 4384.0], [8736.0, -4384.0], [700.0, -59936.0], [1000.0, 58560.0], [0.25, 3.0]]).half()
    pick = torch.randint(0, 5, s.cpu[3].shape[:-1], generator=gen(1))
    s.cpu[3] = par[pick]
    rows = ref.values(s.cpu[1], s.cpu[3], False)[0].abs()
    assert 65520 <= rows.max() < 2 * 65504
    s.to_gpu()
    s.check(kv_cache.fwd(s.cache, s.plan, s.q.cuda()))


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_4_bit_groups_at_the_ends_of_fp16_are_held_finite(dtype):
    """Rows appended with both ends of fp16 in a group: codes and parameters by the formula, held rows the nearest finite
    values, the attention of a token over them finite."""
    s = Step(510, dtype, 4, [40], [0], 2, 2, 64, 16, FULL)
    g = gen(2)
    v = (40000 * torch.randn(40, 2, 64, generator=g)).clamp(-65000, 65000)
    v[..., 3], v[..., 40] = 65504.0, -65504.0
    v[::2, :, 7], v[1::2, :, 50] = -65504.0, 65504.0
    if dtype == BF16:
        v = v.clamp(-65280, 65280)
    s.v = v.to(dtype)
    s.to_gpu()
    _, _, hv = kv_cache.append(s.cache, s.plan, s.k.cuda(), s.v.cuda(), held=True)
    codes, par = ref.quantise(s.v)
    want = (par[..., 1:].double() + par[..., :1].double() * (codes.double() - 8).unflatten(-1, (2, 32))).flatten(-2)
    top = torch.finfo(dtype).max
    assert want.abs().max() > 65504 or dtype == BF16
    assert torch.equal(hv.cpu(), want.clamp(-top, top).to(dtype))
    s.cpu = [t.cpu() for t in (s.cache.k, s.cache.v, s.cache.k_par, s.cache.v_par)]
    s.context[:], s.cu, s.N, s.rows = 39, torch.tensor([0, 1], dtype=torch.int32), 1, [(0, 39)]
    s.q = s.q[:1]
    s.to_gpu()
    s.check(kv_cache.fwd(s.cache, s.plan, s.q.cuda()))


@pytest.mark.parametrize("dtype,d", [(F16, 64), (BF16, 64), (F16, 128)])
@pytest.mark.parametrize("form", list(FORMS))
def test_infinite_values_under_small_weights(form, dtype, d):
    """A value of +-infinity under e^-22 (2^-32), e^-40 and e^-60 of the largest weight is an infinity in the rows that see
    it, in that dimension alone, and nothing elsewhere."""
    new, old, hq, hkv, r = FORMS[form]
    s = Step(520 + d, dtype, 16, new, old, hq, hkv, d, 16, r)
    s.q.zero_()
    s.q[..., 0] = 8.0
    s.cpu[0][..., 0] = 10.0
    p0 = max(0, old[0] - 30)
    for i, (down, x) in enumerate(((22, math.inf), (40, -math.inf), (60, math.inf))):
        at = int(s.table[0, (p0 + i) // 16]), slice(None), (p0 + i) % 16
        s.cpu[0][at][..., 0] = 10.0 - down / 8.0
        s.cpu[1][at][..., 5 + i] = x
    s.to_gpu()
    got = kv_cache.fwd(s.cache, s.plan, s.q.cuda(), scale=1.0).double().cpu()
    other = [e for e in range(d) if e not in (5, 6, 7)]
    seen = 0
    for n, (b, p) in enumerate(s.rows):
        keys = ref.key_set(p, r, 1, None)
        for i, x in enumerate((math.inf, -math.inf, math.inf)):
            if b == 0 and p0 + i in keys and p - p0 > 2 and max(keys) > p0 + 2:
                assert (got[n, :, 5 + i] == x).all(), (n, b, p, i, got[n, :, 5 + i])
                seen += 1
            elif b == 1 or p0 + i not in keys:
                assert torch.isfinite(got[n, :, 5 + i]).all(), (n, b, p, i)
        assert torch.isfinite(got[n][:, other]).all(), (n, b, p)
    assert seen >= 3


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d,hq", [(64, 1), (128, 1), (64, 12), (128, 4)])
def test_small_4_bit_queries_beside_a_large_one(d, hq, dtype):
    """One query value of 1 and, in the other groups, values of 2^-11 (1 + 2^-10) (2^-11 (1 + 2^-7) in bf16) at odd and even
    places: every other key has +7 under the odd and -7 under the even ones, so that its score is 0 as the others' are."""
    x = 2.0 ** -11 * (1 + (2.0 ** -10 if dtype == F16 else 2.0 ** -7))
    s = Step(530, dtype, 4, [1], [255], hq, 1, d, 16, FULL, pages_more=0)
    s.q.zero_()
    s.q[..., 0] = 1.0
    s.q[..., 32:] = x
    codes = torch.full((s.cpu[0].shape[0], 1, 16, d), 8)
    codes[:, :, ::2, 32::2], codes[:, :, ::2, 33::2] = 1, 15
    s.cpu[0] = ref.pack(codes, True)
    s.cpu[2][..., 0], s.cpu[2][..., 1] = 1.0, 0.0
    codes[:, :, ::2], codes[:, :, 1::2] = 15, 0  # values 1.75 and -2: a weight that moves shows
    s.cpu[1], s.cpu[3][..., 0], s.cpu[3][..., 1] = ref.pack(codes, False), 0.25, 0.0
    s.to_gpu()
    scale = 1000.0
    got = kv_cache.fwd(s.cache, s.plan, s.q.cuda(), scale=scale).double().cpu()
    want, by, _ = ref.attend(s.q, s.cpu, s.table, s.rows, s.r, s.dil, None, scale)
    # fp32: a group's sum of q (1024 + c), c < 16, four accumulations that may truncate (2^-23 each) and one rounding when the
    # 1024 is taken off; two such at most move a weight by that share, and its base's share the sum
    score = scale * 5 * 2.0 ** -23 * 1040 * (d - 32) * x
    u = torch.finfo(dtype).eps / 2
    tol = (2.0 ** -10 + 2.0 ** -12) * by + u * want.abs() + score * (by + want.abs())
    assert score < 0.04
    assert ((got - want).abs() <= tol).all(), ((got - want).abs() / tol).max()


CUT = {  # dtype, bits, new, old, hq, hkv, d, page, r, dil, globals: units of single rows that several CTAs share
    "12_on_1": (BF16, 16, [1], [3000], 12, 1, 64, 64, FULL, 1, None),
    "16_on_1_d128": (F16, 16, [1], [2500], 16, 1, 128, 32, FULL, 1, [[0, 9]]),
    "17_on_1": (F16, 16, [1], [2000], 17, 1, 64, 64, FULL, 1, None),
    "34_on_2": (BF16, 16, [1, 1], [1500, 4000], 34, 2, 64, 16, FULL, 1, None),
    "40_on_1_d128": (BF16, 16, [1], [2100], 40, 1, 128, 64, 2000, 1, [[0]]),
    "128_on_1": (F16, 16, [1], [1600], 128, 1, 64, 256, FULL, 1, None),
    "12_on_1_four_d128": (F16, 4, [1], [2500], 12, 1, 128, 32, FULL, 1, None),
    "17_on_1_four": (BF16, 4, [1], [3000], 17, 1, 64, 64, FULL, 1, None),
    "34_on_2_four": (F16, 4, [1, 1], [2600, 1500], 34, 2, 64, 32, FULL, 1, [[3, 0]] * 2),
    "40_on_1_four_d128": (BF16, 4, [1], [3000], 40, 1, 128, 64, FULL, 1, None),
    "dilated": (BF16, 16, [1, 1], [5000, 1200], 8, 4, 64, 64, 1000, [1, 2, 3, 7], [[0, 11, 4000]] * 2),
    "dilated_20_on_2": (F16, 16, [1], [4500], 40, 2, 64, 32, 1200, [1, 3], [[1]]),
    "dilated_four": (F16, 4, [1], [6000], 12, 3, 128, 64, 1500, [1, 2, 4], None),
}


@pytest.mark.parametrize("name", list(CUT))
def test_units_of_many_heads_cut_between_ctas(name):
    s = Step(540 + len(name), *CUT[name]).to_gpu()
    past = s.globals_ is not None and bool((s.globals_ >= s.table.shape[1] * s.page).any())
    assert s.plan.workspace_bytes > 0
    s.plan.buffer.fill_(255)  # entries that the plan does not write: -1
    s.plan.refresh()
    cuts = s.plan.buffer[256 + 640 * 40:256 + 640 * 56].view(torch.int32).view(640, 4)  # (row, unit, last CTA, tile)
    assert (cuts[:, 2] > 0).any()
    got = kv_cache.fwd(s.cache, s.plan, s.q.cuda())
    s.check(got)
    assert torch.equal(got, kv_cache.fwd(s.cache, s.plan, s.q.cuda()))
    assert lf_attn.device_status() == ((5, 1) if past else (0, 0))


def test_flags_of_rows_taken_together():
    """A page outside the cache, then rows behind the table, in tiles: bit 2 and no other."""
    s = Step(550, F16, 16, [280, 21], [40, 10], 4, 2, 64, 16, 25, globals_=[[0, 33], [1, 2]])
    s.table[0, 2], s.table[1, 0] = -5, 1 << 20
    s.to_gpu()
    s.check(kv_cache.fwd(s.cache, s.plan, s.q.cuda()))
    assert lf_attn.device_status() == (5, 4)
    s = Step(551, BF16, 16, [304], [40], 2, 2, 64, 16, 25)
    s.context += 16  # the last 8 rows are behind the table
    s.rows = [(0, 56 + i) if i < 296 else None for i in range(304)]
    s.to_gpu()
    s.check(kv_cache.fwd(s.cache, s.plan, s.q.cuda()))
    assert lf_attn.device_status() == (5, 4)


@pytest.mark.parametrize("cu", [[0, 430, 10, 530, 250], [0, 350, 260, 290, 120], [0, 700, 0, 700, 700]])
def test_no_row_is_one_where_cu_tokens_decreases(cu):
    """Rows that two sequences could claim: none is taken, in tiles or single rows, by the cache or the attention; flagged."""
    for dil in (1, 2):
        s = Step(555, BF16, 16, [200, 300, 150, 50], [10, 0, 40, 3], 2, 2, 64, 16, 30, dil=dil)
        s.cu = torch.tensor(cu, dtype=torch.int32)
        s.to_gpu()
        before = s.cache.k.clone(), s.cache.v.clone()
        q, out = s.q.cuda(), torch.full((700, 2, 64), 2.0, dtype=BF16, device="cuda")
        kv_cache.append(s.cache, s.plan, s.k.cuda(), s.v.cuda())
        kv_cache.fwd(s.cache, s.plan, q, out=out)
        assert (out == 2).all()
        assert torch.equal(s.cache.k, before[0]) and torch.equal(s.cache.v, before[1])
        assert lf_attn.device_status() == (5, 4)
        s.plan.cu_tokens.copy_(torch.tensor([0, 200, 500, 650, 700]))
        s.plan.refresh()
        s.check(kv_cache.fwd(s.cache, s.plan, q))


@pytest.mark.parametrize("call", ["fwd", "append"])
def test_a_plan_outlives_its_use_on_another_stream(call):
    """A plan made on a side stream, used on the current one behind a wait, then dropped: its memory is not given out on the
    side stream before that use."""
    s = Step(580, BF16, 16, [1, 2], [300, 40], 4, 2, 64, 16, FULL).to_gpu()
    q, k, v, side = s.q.cuda(), s.k.cuda(), s.v.cuda(), torch.cuda.Stream()
    plan = kv_cache.Plan(s.cache, s.plan.table, s.plan.cu_tokens, s.plan.context, s.N, s.hq, s.r, stream=side)
    torch.cuda.synchronize()
    size = plan.buffer.numel()
    torch.cuda._sleep(100_000_000)
    got = kv_cache.fwd(s.cache, plan, q) if call == "fwd" else kv_cache.append(s.cache, plan, k, v, q=q)
    del plan
    with torch.cuda.stream(side):
        taken = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert lf_attn.device_status() == (0, 0) and len(taken) == 4
    if call == "fwd":
        s.check(got)
    else:
        assert torch.equal(got, q)


def test_windows_and_dilations_past_32_bits():
    s = Step(560, BF16, 16, [1], [300], 2, 2, 64, 16, FULL).to_gpu()
    q = s.q.cuda()
    plan = lambda r, dil=None: kv_cache.Plan(  # noqa: E731
        s.cache, s.table.cuda(), s.cu.cuda(), s.context.cuda(), 1, 2, r, dil=dil)
    want = kv_cache.fwd(s.cache, s.plan, q)
    for r in (None, (1 << 31) - 1, 1 << 31, 1 << 32, (1 << 32) + 3, 1 << 70):
        assert torch.equal(kv_cache.fwd(s.cache, plan(r), q), want), r
    s.dil = [1 << 20] * 2  # the token's own key alone
    for dil in (1 << 20, (1 << 31) - 1, 1 << 31, (1 << 32) + 1):
        s.check(kv_cache.fwd(s.cache, plan(7, dil), q))


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_strides_of_dimensions_of_one(dtype):
    """One token of a packed row that is no multiple of 16 bytes, and heads of one: strides that nothing steps by."""
    s = Step(570, dtype, 16, [1], [70], 4, 1, 64, 16, 40).to_gpu()
    wide = torch.zeros(2, 6 * 64 + 1, dtype=dtype)
    wide[0, :256], wide[0, 256:320], wide[0, 320:384] = s.q.flatten(), s.k.flatten(), s.v.flatten()
    wide = wide.cuda()
    q, k, v = (torch.as_strided(wide, (1, h, 64), (385, 64, 1), 64 * a) for h, a in ((4, 0), (1, 4), (1, 5)))
    s.check(kv_cache.fwd(s.cache, s.plan, q))
    f = rotary.freqs(64, device="cuda")
    got = kv_cache.append(s.cache, s.plan, k, v, q=q, freqs=f)
    want = ref.turn(s.q.double(), torch.tensor([70])[:, None], f.tolist())
    assert ((got.double().cpu() - want).abs() <= turn_tolerance(s.q.double(), want, dtype, 1.0)).all()
    far = torch.as_strided(wide, (1, 1, 64), (1 << 40, 1 << 41, 1))
    other = Step(571, dtype, 16, [1], [70], 1, 1, 64, 16, 40).to_gpu()
    other.q = far.cpu()
    other.check(kv_cache.fwd(other.cache, other.plan, far))
    one = torch.as_strided(wide, (1, 1, 1, 64), (1 << 41, 1 << 40, 1 << 39, 1))
    got = rotary.fwd(one, freqs=f, pos=torch.tensor([9], dtype=torch.int32, device="cuda"))[0]
    want = ref.turn(one.double().cpu(), torch.tensor([9]), f.tolist())
    assert ((got.double().cpu() - want).abs() <= turn_tolerance(one.double().cpu(), want, dtype, 1.0)).all()
