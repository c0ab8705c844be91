"""The paged cache at the ends of its types and shapes, against the definitions in 64 bits."""
import pytest
import torch

from sparse_long_sequence_fwd_b200 import kv_cache
from tests import cache_ref as ref
from tests.test_gpu_cache import BF16, F16, FULL, Step, _lib, _no_flags, gen  # noqa: F401

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
