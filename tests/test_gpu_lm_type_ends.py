"""Finite values next to the ends of their type, through a cache of 8-bit codes: what was finite
when it was stored is finite when it is read."""
import math

import pytest
import torch

import lm_ref8
from ctc_prefix_beam_amd import lm

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]
CODES = [torch.int8, torch.float8_e4m3fn]


def stored(x, code, page=8):
    """x (tokens, heads, dim) in a cache, a page to each token: the slots and the cache."""
    T, H, D = x.shape
    c = [torch.zeros((T, page, H, D), dtype=torch.int8, device="cuda").view(code) for _ in range(2)]
    s = [torch.zeros((T, H), device="cuda") for _ in range(2)]
    slots = torch.arange(T, dtype=torch.int32, device="cuda") * page
    lm.cache_store8(x, -x, slots, *c, *s)
    return slots, (*c, *s)


def ends(dtype, D):
    """Rows whose largest value is the type's largest one, or shares of it down to a half."""
    share = torch.tensor([1, 1 - 2.0 ** -8, 0.995, 0.99, 0.98, 0.95, 0.9, 0.75, 0.51, 0.5])
    x = (share.double() * torch.finfo(dtype).max).to(dtype)
    x = x[:, None, None].repeat(1, 2, D)
    x[:, 1] *= -1
    x[..., 1::3] *= 0.25
    return x.cuda()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("D", [64, 5])   # pieces of 16 bytes, and single values
def test_what_is_finite_is_read_back_finite(dtype, code, D):
    """The largest value stands for itself (|clamped code - x| <= |code - x|): off by half a step
    at most, which is u / 2 for whole numbers and 1/16 of the value for e4m3's three bits."""
    x = ends(dtype, D)
    slots, cache = stored(x, code)
    assert torch.isfinite(cache[2]).all()
    k, v = lm.cache_load8(slots, *cache, dtype=dtype)
    assert torch.isfinite(k).all() and torch.equal(v, -k)
    # the nearest code stands for more than the type holds: what this is about
    over = lm_ref8.values(cache[0])[:, 0].abs() * cache[2].cpu().double()[..., None]
    assert (over > torch.finfo(dtype).max).any()
    off = (k.double() - x.double()).abs()
    half = cache[2].double()[..., None] / 2 if code == torch.int8 else x.double().abs() / 16
    # (and the rounding to the type)
    assert (off <= half * (1 + 2.0 ** -20) + lm_ref8.HALF[dtype] * x.double().abs()).all()


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("D", [64, 5])
def test_a_narrower_type_ends_at_its_largest_value(code, D):
    x = torch.full((3, 1, D), 1e30, device="cuda")
    x[1], x[2] = 100000.0, 60000.0
    x[:, :, ::2] *= -1
    slots, cache = stored(x, code)
    k, _ = lm.cache_load8(slots, *cache, dtype=torch.float16)
    assert torch.equal(k[:2].float(), x[:2].sign() * 65504.0)
    assert ((k[2].float() - x[2]).abs() <= 60000 / 16).all()
    k, _ = lm.cache_load8(slots, *cache, dtype=torch.bfloat16)
    assert torch.isfinite(k).all() and (k[0].float().abs() > 9e29).all()


@pytest.mark.parametrize("D", [64, 5])
def test_what_is_not_finite_stays_so(D):
    x = ends(torch.float32, D)[:3].contiguous()
    x[1, 0, 2] = math.inf
    x[2, 1, 0] = math.nan
    slots, cache = stored(x, torch.int8)
    k, _ = lm.cache_load8(slots, *cache, dtype=torch.float16)
    bad = torch.zeros((3, 2), dtype=torch.bool, device="cuda")
    bad[1, 0] = bad[2, 1] = True
    assert torch.equal(torch.isnan(k).all(-1), bad) and torch.equal(torch.isnan(k).any(-1), bad)
    # a code that is no number, beside one that is, under a large scale
    slots, cache = stored(ends(torch.float16, D)[:1].contiguous(), torch.float8_e4m3fn)
    cache[0].view(torch.uint8)[0, 0, 0, 1] = 127
    k, _ = lm.cache_load8(slots, *cache, dtype=torch.float16)
    assert torch.isnan(k[0, 0, 1]) and torch.isfinite(k[0, 0, 0]) and torch.isfinite(k[0, 1]).all()
    # and a scale that was set to infinity
    cache[2].fill_(math.inf)
    k, _ = lm.cache_load8(slots, *cache, dtype=torch.float16)
    assert not torch.isfinite(k).any()


@pytest.mark.parametrize("D", [64, 5])
def test_scales_below_zero_turn_the_signs(D):
    """A store makes none, but a load takes any."""
    slots, cache = stored(ends(torch.float16, D), torch.int8)
    k, v = lm.cache_load8(slots, *cache, dtype=torch.float16)
    got = lm.cache_load8(slots, cache[0], cache[1], -cache[2], -cache[3], dtype=torch.float16)
    assert torch.equal(got[0], -k) and torch.equal(got[1], -v) and torch.isfinite(k).all()


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows,n", [(4, 8), (3000, 8), (2, 6000)])   # each launch form
def test_attention_over_values_at_the_end_of_f16(code, D, rows, n):
    """Every token's values lie between 0.99 and 1 of the largest one, with the same signs: so do the
    results.  Codes are half a step off (u / 2, and 1/16 for e4m3's), never past the end."""
    page, kept = 8, -(-n // 8)
    g = torch.Generator().manual_seed(D)
    v = (65504 * (0.99 + 0.01 * torch.rand((kept * page, 1, D), generator=g))).to(torch.float16)
    v[0] = 65504
    v[..., ::2] *= -1
    v = v.cuda()
    kc = torch.zeros((kept, page, 1, D), dtype=torch.int8, device="cuda").view(code)
    vc, ks, vs = kc.clone(), torch.zeros((kept, 1), device="cuda"), torch.zeros((kept, 1), device="cuda")
    slots = torch.arange(kept * page, dtype=torch.int32, device="cuda")
    lm.cache_store8(torch.zeros_like(v), v, slots, kc, vc, ks, vs)
    tables = torch.arange(kept, dtype=torch.int32, device="cuda").repeat(rows, 1)
    lens = torch.full((rows,), n, dtype=torch.int32, device="cuda")
    lens[0] = 1
    q = torch.randn((rows, 2, D), device="cuda").to(torch.float16)
    out, _ = lm.attention8(q, kc, vc, ks, vs, tables, lens)
    assert torch.isfinite(out).all()
    sign = v[0, 0].sign().float()
    assert (out.float() * sign <= 65504).all()
    assert (out.float() * sign >= 65504 * 0.99 * (1 - 1 / 16 - 2.0 ** -10)).all()
    assert (out[0].float() == 65504 * sign).all()
