"""The store to a cache of 8-bit codes and the way back, against 64 bits: codes, scales and
values are equal."""
import math

import pytest
import torch

import lm_ref8
from ctc_prefix_beam_amd import lm

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]
CODES = [torch.int8, torch.float8_e4m3fn]


def cache(pages, page, H, D, code, order="thd", seed=0, scales="some"):
    """(codes, scales): what earlier tokens left; e4m3 codes of every kind but NaN."""
    g = torch.Generator().manual_seed(seed)
    shape = (pages, page, H, D) if order == "thd" else (pages, H, page, D)
    b = torch.randint(0, 256, shape, generator=g, dtype=torch.int32).to(torch.uint8)
    if code == torch.int8:
        b[b == 128] = 0
    else:
        b[(b & 127) == 127] = 0
    c = b.cuda().view(code)
    if order == "htd":
        c = c.transpose(1, 2)
    e = torch.randint(-9, -3, (pages, H), generator=g)
    s = torch.exp2(e.float()) if scales == "some" else torch.zeros((pages, H))
    return c, s.cuda()


def slots_of(counts, held, page, seed=0, spare=2):
    """Slots of counts[r] new tokens behind held[r] in pages of their own, and the page count."""
    g = torch.Generator().manual_seed(seed + 1)
    need = [-(-(h + n) // page) for h, n in zip(held, counts)]
    ids = torch.randperm(sum(need) + spare, generator=g).tolist()
    slots, at = [], 0
    for n, h, k in zip(counts, held, need):
        slots += [ids[at + p // page] * page + p % page for p in range(h, h + n)]
        at += k
    return torch.tensor(slots, dtype=torch.int32), sum(need) + spare


def check(x, y, slots, kc, ks, vc, vs, **kw):
    """Stores and compares codes, scales and what is read back."""
    want = [lm_ref8.store(a, slots, c, s) for a, c, s in ((x, kc, ks), (y, vc, vs))]
    lm.cache_store8(x, y, slots, kc, vc, ks, vs, **kw)
    for (vals, scales), c, s in zip(want, (kc, vc), (ks, vs)):
        assert torch.equal(s.cpu().double().nan_to_num(-1), scales.nan_to_num(-1))
        assert torch.equal(lm_ref8.values(c), vals)
    for dtype in (x.dtype, torch.bfloat16):
        k, v = lm.cache_load8(slots, kc, vc, ks, vs, dtype)
        assert k.dtype == dtype
        for got, c, s in ((k, kc, ks), (v, vc, vs)):
            assert torch.equal(got.cpu().nan_to_num(-1),
                               lm_ref8.load(slots, c, s, dtype).nan_to_num(-1))


def random(slots, H, D, dtype, seed=0, size=1.0):
    g = torch.Generator().manual_seed(seed + 2)
    T = slots.numel()
    x = torch.randn((2, T, H, D), generator=g) * size
    x = x * torch.exp2(torch.randint(-3, 4, (2, T, 1, 1), generator=g).float())
    return x.to(dtype).cuda().unbind(0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("D", [1, 8, 20, 64, 72, 128, 200, 256])
def test_head_dims(dtype, code, D):
    slots, pages = slots_of([1, 5, 16, 33, 0, 2], [0, 3, 0, 9, 1, 15], 16)
    x, y = random(slots, 3, D, dtype, D)
    check(x, y, slots.cuda(), *cache(pages, 16, 3, D, code), *cache(pages, 16, 3, D, code, seed=5))


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("page", [4, 8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("order", ["thd", "htd"])
@pytest.mark.parametrize("counts,held", [([1] * 9, list(range(9))), ([300, 7, 1, 70], [0, 3, 64, 1])])
def test_pages_and_orders(code, page, order, counts, held):
    slots, pages = slots_of(counts, [h % page for h in held], page)
    x, y = random(slots, 2, 64, torch.bfloat16, page)
    check(x, y, slots.cuda(), *cache(pages, page, 2, 64, code, order),
          *cache(pages, page, 2, 64, code, order, 5))


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("chunks", [False, True])
def test_tokens_without_a_slot(code, dtype, chunks):
    """Between the tokens of a page, in front of them and behind, short and long stretches; with
    many heads the store goes by chunks of tokens.  What they hold is not looked at."""
    H = 300 if chunks else 2
    slots, pages = slots_of([40, 3, 50, 20, 1], [0, 2, 5, 0, 7], 16)
    g = torch.Generator().manual_seed(3)
    slots[torch.rand(slots.numel(), generator=g) < 0.3] = -1
    gap = torch.full((150,), -1, dtype=torch.int32)
    past = torch.full((3,), pages * 16, dtype=torch.int32)
    slots = torch.cat((gap[:2], slots[:50], gap, slots[50:60], past, slots[60:], gap[:70]))
    x, y = random(slots, H, 16, dtype)
    off = ((slots < 0) | (slots >= pages * 16)).cuda()
    x[off], y[off] = math.nan, math.inf
    check(x, y, slots.cuda(), *cache(pages, 16, H, 16, code), *cache(pages, 16, H, 16, code, seed=5))


@pytest.mark.parametrize("code", CODES)
def test_a_page_filled_token_by_token(code):
    """Its scale grows with the largest value and never shrinks.  Each rescaling rounds by half a
    step, of which all earlier ones are at most a half, a quarter and so on: less than one step
    in all; e4m3 codes that stay normal are only shifted."""
    g = torch.Generator().manual_seed(8)
    H, D, page = 3, 64, 16
    x = torch.randn((2, 2 * page, H, D), generator=g)
    x = (x * torch.exp2(torch.linspace(-2, 3, 2 * page))[:, None, None]).cuda()
    kc, ks = cache(2, page, H, D, code)
    vc, vs = cache(2, page, H, D, code, seed=1)
    last = torch.zeros_like(ks)
    for t in range(2 * page):
        check(x[0, t:t + 1], x[1, t:t + 1], torch.tensor([t], dtype=torch.int32, device="cuda"), kc,
              ks, vc, vs)
        assert (ks[:t // page + 1] >= last[:t // page + 1])[t // page].all() or t % page == 0
        last = ks.clone()
    slots = torch.arange(2 * page, dtype=torch.int32, device="cuda")
    for got, want, s in zip(lm.cache_load8(slots, kc, vc, ks, vs, torch.float32), x, (ks, vs)):
        step = s.repeat_interleave(page, 0)[..., None].expand_as(want)
        if code == torch.float8_e4m3fn:
            # half a step of the value's own binade, or one of the smallest codes'
            e = torch.floor(torch.log2((want / step).abs().clamp(min=2.0 ** -6)))
            step = torch.maximum(step * torch.exp2(e - 3) / 2, step * 2.0 ** -9)
        assert ((got - want).abs() <= step * (1 + 2.0 ** -20)).all()


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", TYPES)
def test_borders_of_the_scale(code, dtype):
    """Largest values at, just below and just above top times a power of two, at a type's ends,
    ties between codes, zeros, infinities and NaN."""
    top = lm_ref8.TOP[code]
    info = torch.finfo(dtype)
    above = float(torch.nextafter(torch.tensor(float(top)).to(dtype), torch.tensor(9e9).to(dtype)))
    big = 2.0 ** 100 if dtype != torch.float16 else 2.0 ** 6
    rows = [[top, 0.5, 1.5, 2.5], [above, 0.5, 1.5, 2.5], [2 * top, 1, 3, 5],
            [info.max, 1, 0, -info.max], [info.tiny, 0, -info.tiny, info.smallest_normal],
            [info.smallest_normal * 2.0 ** -3, 0, 0, 0], [0, 0, 0, 0], [-0.0, 0, 0, 0],
            [math.inf, 1, 2, 3], [1, -math.inf, 2, 3], [1, math.nan, 2, 3], [-top, -0.5, -1.5, 0.25],
            [top * big, big * 1.5, 2.5 * big, 0.49 * big], [17, 19, 0.001953125 * 9, 21]]
    x = torch.tensor(rows).to(dtype).cuda()[:, None].repeat(1, 2, 2)
    slots = torch.arange(len(rows), dtype=torch.int32, device="cuda") * 8
    kc, ks = cache(len(rows), 8, 2, 8, code)
    vc, vs = cache(len(rows), 8, 2, 8, code, seed=1)
    check(x, x.flip(0), slots, kc, ks, vc, vs)
    # and as the second token of the pages, with scales that are there
    check(x.roll(3, 0), x, slots + 1, kc, ks, vc, vs)
    bad = ~torch.isfinite(x.roll(3, 0)).all(-1) | ~torch.isfinite(x).all(-1)
    assert torch.equal(torch.isnan(ks), bad)
    # a page that begins anew forgets what was not finite
    check(torch.ones_like(x), torch.ones_like(x), slots, kc, ks, vc, vs)
    assert torch.isfinite(ks).all() and torch.isfinite(vs).all()


def test_scales_of_zero_and_of_any_size():
    """Pages that nothing was stored to yet, and scales that are no power of two."""
    slots = torch.tensor([3, 9, 17], dtype=torch.int32, device="cuda")
    kc, ks = cache(3, 8, 1, 16, torch.int8, scales="none")
    vc, vs = cache(3, 8, 1, 16, torch.int8)
    kc.zero_()
    x = torch.zeros((3, 1, 16), device="cuda")
    x[1] = 5.0
    check(x, x, slots, kc, ks, vc, vs)
    assert ks.flatten().tolist() == [0.0, 2.0 ** -4, 0.0]
    ks[1] = 0.3
    lm.cache_store8(x, x, slots, kc, vc, ks, vs)
    assert abs(float(ks[1, 0]) - 0.3) < 1e-7 and kc[1, 1].unique().tolist() == [17]   # 5 / 0.3


def test_strided_inputs_and_scales():
    slots, pages = slots_of([1, 20, 9], [0, 3, 15], 16)
    g = torch.Generator().manual_seed(0)
    fused = torch.randn((30, 7, 65), generator=g).to(torch.float16).cuda()
    x, y = fused[:, 1:3, 1:], fused[:, 4:6, :64]
    big = torch.zeros((pages, 16, 5, 70), dtype=torch.int8, device="cuda")
    scales = torch.zeros((pages, 3, 2), device="cuda")
    check(x, y, slots.cuda(), big[:, :, 1:3, 3:67], scales[:, 1:, 0], big[:, :, 3:5, :64],
          scales[:, 1:, 1])
    assert (big[:, :, 0] == 0).all() and (big[..., 67:] == 0).all()
    assert (big[:, :, 1:3, :3] == 0).all() and (scales[:, 0] == 0).all()
    one = fused[:1, :1].expand(30, 2, 65)[..., :64]   # inputs may be expanded
    check(one, one, slots.cuda(), *cache(pages, 16, 2, 64, torch.int8),
          *cache(pages, 16, 2, 64, torch.int8, seed=1))


def test_many_tokens():
    """Prompts beside single tokens, in one call."""
    g = torch.Generator().manual_seed(0)
    counts = torch.randint(0, 90, (700,), generator=g).tolist()
    held = torch.randint(0, 40, (700,), generator=g).tolist()
    slots, pages = slots_of(counts, [h % 16 for h in held], 16)
    x, y = random(slots, 2, 64, torch.bfloat16)
    check(x, y, slots.cuda(), *cache(pages, 16, 2, 64, torch.int8),
          *cache(pages, 16, 2, 64, torch.int8, seed=1))


@pytest.mark.parametrize("page,D,dtype,code", [
    (32, 128, torch.bfloat16, torch.int8), (64, 128, torch.float16, torch.float8_e4m3fn),
    (16, 128, torch.float32, torch.int8), (256, 64, torch.bfloat16, torch.float8_e4m3fn),
    (256, 256, torch.float32, torch.int8), (32, 20, torch.bfloat16, torch.int8),
    (64, 36, torch.float32, torch.float8_e4m3fn), (128, 13, torch.float16, torch.int8)])
def test_many_tokens_in_larger_pages(page, D, dtype, code):
    """Pages whose values take several waves' registers, or more; begun, gone on with and filled
    over in one call, among single tokens and tokens without a slot."""
    H = 60
    g = torch.Generator().manual_seed(page + D)
    counts = torch.randint(0, 130, (12,), generator=g).tolist() + [1] * 9
    held = torch.randint(0, page, (21,), generator=g).tolist()
    slots, pages = slots_of(counts, held, page)
    slots[torch.rand(slots.numel(), generator=g) < 0.05] = -1
    assert slots.numel() * H * 2 > 1 << 16   # not a wave to each token
    x, y = random(slots, H, D, dtype)
    check(x, y, slots.cuda(), *cache(pages, page, H, D, code, "htd"),
          *cache(pages, page, H, D, code, "thd", seed=1))


@pytest.mark.parametrize("page,D,dtype,code", [
    (16, 64, torch.bfloat16, torch.int8), (16, 64, torch.float16, torch.float8_e4m3fn),
    (8, 128, torch.float16, torch.int8), (16, 32, torch.float32, torch.float8_e4m3fn),
    (4, 256, torch.bfloat16, torch.float8_e4m3fn), (4, 20, torch.bfloat16, torch.int8),
    (8, 13, torch.float32, torch.int8)])
def test_many_tokens_in_small_pages(page, D, dtype, code):
    """Pages whose keys and values one wave stores together: begun, gone on with, with tokens
    without a slot between (a run of more tokens than the page has slots), and keys or values
    alone that raise a scale or are not finite."""
    H = 60
    g = torch.Generator().manual_seed(page + D)
    counts = torch.randint(0, 130, (16,), generator=g).tolist() + [1] * 30
    held = torch.randint(0, page, (46,), generator=g).tolist()
    slots, pages = slots_of(counts, held, page)
    gaps = torch.rand(slots.numel(), generator=g) < 0.4
    gaps[400:] = False
    slots = torch.stack((slots, torch.full_like(slots, -1)), 1).flatten()[
        torch.stack((torch.ones_like(gaps), gaps), 1).flatten()]
    assert slots.numel() * H * 2 > 1 << 16   # not a wave to each token
    x, y = (t.clone() for t in random(slots, H, D, dtype))
    x[::7, 3] *= 512
    y[::11, 4] *= 512
    x[100, 5, D - 1], y[200, 6, 0] = math.nan, math.inf
    check(x, y, slots.cuda(), *cache(pages, page, H, D, code, "htd"),
          *cache(pages, page, H, D, code, "thd", seed=1))


def test_no_tokens_and_a_stream_of_its_own():
    kc, ks = cache(3, 16, 2, 64, torch.int8)
    vc, vs = cache(3, 16, 2, 64, torch.int8)
    none = torch.zeros((0, 2, 64), device="cuda")
    lm.cache_store8(none, none, torch.zeros(0, dtype=torch.int32, device="cuda"), kc, vc, ks, vs)
    k, v = lm.cache_load8(torch.zeros(0, dtype=torch.int32, device="cuda"), kc, vc, ks, vs)
    assert k.shape == v.shape == (0, 2, 64)
    slots = torch.tensor([0, 1, 5], dtype=torch.int32, device="cuda")
    x, y = random(slots, 2, 64, torch.float32)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    want = lm_ref8.store(x, slots, kc, ks)
    lm.cache_store8(x, y, slots, kc, vc, ks, vs, stream=side)
    k, _ = lm.cache_load8(slots, kc, vc, ks, vs, torch.float32, stream=side)
    side.synchronize()
    assert torch.equal(lm_ref8.values(kc), want[0])
    assert torch.equal(k.cpu(), lm_ref8.load(slots, kc, ks, torch.float32))


def test_a_cache_past_32_bits():
    """Pages whose codes lie more than 2^32 bytes behind the first one's."""
    pages, page, H, D = 66000, 256, 2, 128
    kc = torch.zeros((pages, page, H, D), dtype=torch.int8, device="cuda")
    assert kc.numel() > 1 << 32
    ks = torch.zeros((pages, H), device="cuda")
    x = torch.randn((4, H, D), device="cuda")
    slots = torch.tensor([0, 256 * 40000, 256 * 65999, 256 * 65999 + 1], dtype=torch.int32,
                         device="cuda")
    vc, vs = kc.clone(), ks.clone()
    lm.cache_store8(x, -x, slots, kc, vc, ks, vs)
    k, v = lm.cache_load8(slots, kc, vc, ks, vs, torch.float32)
    s = ks[(slots // 256).long()][..., None]
    assert (s > 0).all() and ((k - x).abs() <= s / 2).all() and torch.equal(v, -k)
    assert int((kc != 0).any(-1).sum()) == 4 * H


def test_refusals():
    kc, ks = cache(3, 16, 2, 64, torch.int8)
    x = torch.zeros((2, 2, 64), device="cuda")
    s = torch.zeros(2, dtype=torch.int32, device="cuda")
    good = dict(k=x, v=x, slots=s, k_cache=kc, v_cache=kc.clone(), k_scale=ks, v_scale=ks.clone())
    for kw in (dict(k_cache=kc.float()), dict(v_cache=kc.view(torch.float8_e4m3fn)),
               dict(k_scale=ks.double()), dict(k_scale=ks[:2]), dict(v_scale=ks[:, :1]),
               dict(k_scale=ks[:1].expand(3, 2)), dict(k_cache=kc[:1].expand(3, 16, 2, 64)),
               dict(k=x.double()), dict(v=x[:1]), dict(slots=s.long()), dict(k=x[:, :1], v=x[:, :1]),
               dict(k=x.clone().requires_grad_()), dict(k_scale=ks.cpu()), dict(k=x.cpu())):
        with pytest.raises((ValueError, TypeError)):
            lm.cache_store8(**{**good, **kw})
    for kw in (dict(dtype=torch.int8), dict(dtype=torch.float64)):
        with pytest.raises(ValueError, match="dtype"):
            lm.cache_load8(s, kc, kc, ks, ks, **kw)
    lm.cache_load8(s, kc[:1].expand(3, 16, 2, 64), kc, ks[:1].expand(3, 2), ks)   # read, they may be
