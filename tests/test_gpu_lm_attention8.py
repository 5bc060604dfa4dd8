"""Attention over a cache of 8-bit codes, against float64 on the values they stand for."""
import math

import pytest
import torch

import lm_ref
import lm_ref8
from ctc_prefix_beam_amd import lm

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]
CODES = [torch.int8, torch.float8_e4m3fn]


def make(lengths, Hq, Hkv, D, dtype, code, page, order="thd", seed=0, width=None, spread=2):
    """q, codes, scales (2^-spread .. 2^spread about what makes values of one), tables, lengths.
    Slots that no request owns hold NaN where codes can, the largest code where not, and pages
    that none owns have NaN scales."""
    g = torch.Generator().manual_seed(seed)
    have = [-(-max(n, 0) // page) for n in lengths]
    pages = sum(have) + 2
    perm = torch.randperm(pages, generator=g).tolist()
    width = max(have + [1]) if width is None else width
    tables = torch.full((len(lengths), width), -1, dtype=torch.int32)
    used = torch.zeros((pages, page), dtype=torch.bool)
    at = 0
    for r, k in enumerate(have):
        for j in range(k):
            tables[r, j] = perm[at]
            used[perm[at], :max(0, min(page, lengths[r] - j * page))] = True
            at += 1
    cache = []
    for _ in range(2):
        c = torch.randn((pages, page, Hkv, D), generator=g) * (lm_ref8.TOP[code] / 4)
        c = c.clamp(-lm_ref8.TOP[code], lm_ref8.TOP[code])
        c = (c.round() if code == torch.int8 else c).to(code)
        b = c.view(torch.uint8)
        b[~used] = 127
        e = torch.randint(-spread, spread + 1, (pages, Hkv), generator=g).float()
        s = torch.exp2(e) * 4 / 2.0 ** round(math.log2(lm_ref8.TOP[code]))
        s[~used.any(1)] = math.nan
        if order == "htd":
            b = b.transpose(1, 2).contiguous().transpose(1, 2)
        dev = b.cuda().view(code)
        assert dev.stride() == b.stride()
        cache.append((dev, s.cuda()))
    q = 2 * torch.randn((len(lengths), Hq, D), generator=g)
    (kc, ks), (vc, vs) = cache
    return (q.to(dtype).cuda(), kc, vc, ks, vs, tables.cuda(),
            torch.tensor(lengths, dtype=torch.int32).cuda())


def real(c, s):
    return lm_ref8.values(c) * s.cpu().double()[:, None, :, None]


def check(q, kc, vc, ks, vs, tables, lens, page, scale=None, window=0, **kw):
    """The tolerances are those of the 16- and 32-bit caches: codes are exact, and so is their way
    into the products; q in two f16 values is off by 2^-23 of itself (f32) or 2^-39 of the largest
    (bf16), inside the D + 4 roundings that a score is given, and a score's factor adds
    two; weights in two f16 values are off by 2^-22, of 2^-16 given."""
    out, lse = lm.attention8(q, kc, vc, ks, vs, tables, lens, scale=scale, window=window, **kw)
    s = q.shape[2] ** -0.5 if scale is None else scale
    wo, wl, to, tl = lm_ref.attention(q, real(kc, ks), real(vc, vs), tables, lens, s, window, page)
    out, lse = out.cpu().double(), lse.cpu().double()
    assert torch.isfinite(out).all()
    assert ((out - wo).abs() <= to).all(), float(((out - wo).abs() - to).max())
    dead = wl == -math.inf
    assert torch.equal(lse == -math.inf, dead)
    assert ((lse - wl).abs()[~dead] <= tl[~dead]).all()
    return out


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("D", [16, 48, 64, 80, 96, 128, 144, 192, 256])
def test_head_dims(dtype, code, D):
    check(*make([0, 1, 31, 32, 33, 150], 4, 2, D, dtype, code, 16, seed=D), 16)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (5, 1), (8, 1), (16, 1), (17, 1), (40, 2),
                                    (64, 2), (12, 4)])
def test_head_groups(dtype, Hq, Hkv):
    for code in CODES:
        check(*make([1, 0, 70, 300], Hq, Hkv, 64, dtype, code, 16, seed=Hq), 16)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("page", [4, 8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("order", ["thd", "htd"])
def test_pages_and_orders(dtype, page, order):
    for code in CODES:
        check(*make([1, 3, 4, 5, 127, 128, 129, 513, 0, 1000], 6, 3, 64, dtype, code, page, order,
                    page), page)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("n", [1, 128, 257, 4096, 20011])
def test_one_request_split_over_its_length(dtype, code, n):
    check(*make([n], 8, 2, 128, dtype, code, 16, seed=n), 16)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("window", [1, 2, 15, 33, 200, 5000])
def test_window(dtype, window):
    for code in CODES:
        check(*make([0, 1, 30, 64, 333, 4000], 4, 2, 64, dtype, code, 8, seed=window), 8,
              window=window)


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_rows(code, D):
    lens = [(7 * r) % 90 for r in range(1500)]
    check(*make(lens, 4, 2, D, torch.bfloat16, code, 16), 16)
    check(*make(lens, 4, 2, D, torch.float32, code, 16), 16, window=21)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [48, 64, 128, 256])
@pytest.mark.parametrize("width", [70, 140, 2000])
@pytest.mark.parametrize("window", [0, 37, 600])
def test_short_rows_in_tables_of_any_width(dtype, D, width, window):
    lens = [0, 1, 3, 16, 17, 0, 500, 64, 1100, 255]
    for code in CODES:
        check(*make(lens, 6, 3, D, dtype, code, 16, seed=D, width=width), 16, window=window)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group", [1, 2, 3, 5, 16, 17, 40])
@pytest.mark.parametrize("D", [64, 80, 128, 256])
def test_parts_of_split_rows(dtype, group, D):
    """Ranges with every head group, joined from one part and from many."""
    check(*make([3000, 1, 900, 5000], group, 1, D, dtype, torch.int8, 16, seed=group), 16)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("code", CODES)
def test_scales_far_apart(dtype, code):
    """Pages whose scales span 2^60, keys and values."""
    q, kc, vc, ks, vs, tables, lens = make([100, 700, 3000], 4, 2, 64, dtype, code, 16, spread=0)
    g = torch.Generator().manual_seed(0)
    e = torch.randint(-30, 31, vs.shape, generator=g).float()
    small = torch.exp2(e - 45).cuda()   # values far below a float32 of one
    if dtype != torch.float16:   # (f16 results end at 65504)
        check(q, kc, vc, ks, vs * torch.exp2(e).cuda(), tables, lens, 16)
    check(q, kc, vc, ks, vs * small, tables, lens, 16)
    check(q, kc, vc, ks * torch.exp2(-e.abs()).cuda(), vs, tables, lens, 16)


def test_weight_on_small_values_beside_large_ones():
    """All probability on a page of tiny values, next to a huge page that has none: its digits are
    those of the tiny values (relative to them)."""
    for code in CODES:
        for dtype in TYPES[::2]:
            q, kc, vc, ks, vs, tables, lens = make([64], 1, 1, 64, dtype, code, 32, spread=0)
            q.fill_(1.0)
            kc.view(torch.uint8)[:] = 127 if code == torch.int8 else 126
            ks.fill_(0.05)
            p0, p1 = tables[0].tolist()
            kc[p1] = (-kc[p1].float()).to(code)    # scores some hundred below the others'
            vs[p0], vs[p1] = 2.0 ** -40, 2.0 ** 20
            for t in (tables, tables.flip(1)):     # the tiny page first, and last
                out, _ = lm.attention8(q, kc, vc, ks, vs, t, lens)
                want = real(vc, vs)[p0, :, 0].mean(0)
                tol = 2.0 ** -16 * float(real(vc, vs)[p0].abs().max())
                tol = tol + lm_ref8.HALF[dtype] * want.abs()
                assert ((out[0, 0].cpu().double() - want).abs() <= tol).all()


def test_scores_of_any_size():
    q, kc, vc, ks, vs, tables, lens = make([200, 64, 50], 2, 1, 64, torch.float32, torch.int8, 16)
    check(q * 300, kc, vc, ks, vs, tables, lens, 16)     # one token takes all
    check(q * 0, kc, vc, ks, vs, tables, lens, 16)       # all tokens alike
    check(q * 2.0 ** -100, kc, vc, ks, vs, tables, lens, 16)
    check(q * 2.0 ** 90, kc, vc, ks, vs, tables, lens, 16, scale=2.0 ** -92)
    check(q, kc, vc, ks * 0, vs, tables, lens, 16)       # pages of scale 0: scores of 0
    check(q, kc, vc, ks, vs * 0, tables, lens, 16)
    check(q, kc, vc, ks, vs, tables, lens, 16, scale=-0.3)
    one = q.clone()
    one[:, :, 1:] *= 2.0 ** -30                          # one large number in each row
    check(one, kc, vc, ks, vs, tables, lens, 16)


@pytest.mark.parametrize("dtype", TYPES)
def test_a_page_that_is_not_finite_is_its_rows_alone(dtype):
    q, kc, vc, ks, vs, tables, lens = make([100, 40, 300], 2, 1, 64, dtype, torch.int8, 16)
    want, wl = lm.attention8(q, kc, vc, ks, vs, tables, lens)
    for s in (ks, vs):
        t = s.clone()
        t[tables[1, 1].long()] = math.nan
        out, lse = lm.attention8(q, kc, vc, *((t, vs) if s is ks else (ks, t)), tables, lens)
        assert torch.isnan(out[1]).all()
        assert torch.equal(out[0], want[0]) and torch.equal(out[2], want[2])
        assert torch.equal(lse[::2], wl[::2]) and torch.isnan(lse[1]).any() == (s is ks)
    q[0, 1, 5] = math.nan
    out, lse = lm.attention8(q, kc, vc, ks, vs, tables, lens)
    assert torch.isnan(out[0, 1]).all()
    assert torch.equal(out[0, 0], want[0, 0]) and torch.equal(out[1:], want[1:])


def test_strided_q_out_and_scales():
    q, kc, vc, ks, vs, tables, lens = make([40, 9], 4, 2, 64, torch.float16, torch.int8, 16)
    fused = torch.zeros((2, 8, 65), dtype=q.dtype, device="cuda")
    fused[:, 2:6, 1:] = q
    big = torch.full((2, 9, 70), 3.0, dtype=q.dtype, device="cuda")
    both = torch.stack((ks, vs), -1)
    want, _ = lm.attention8(q, kc, vc, ks, vs, tables, lens)
    got, _ = lm.attention8(fused[:, 2:6, 1:], kc, vc, both[..., 0], both[..., 1], tables, lens,
                           out=big[:, 1:5, 3:67])
    assert torch.equal(got, want)
    assert (big[:, 0] == 3).all() and (big[:, 5:] == 3).all() and (big[:, :, :3] == 3).all()


@pytest.mark.parametrize("lens", [[300] * 3, [3000, 17, 0], [(9 * r) % 70 for r in range(900)]])
def test_out_in_place_of_q(lens):
    a = make(lens, 40, 2, 64, torch.bfloat16, torch.int8, 16)
    want, _ = lm.attention8(*a)
    q = a[0].clone()
    lm.attention8(q, *a[1:], out=q)
    assert torch.equal(q, want)
    big = torch.zeros((q.shape[0] + 1, 40, 64), dtype=q.dtype, device="cuda")
    with pytest.raises(ValueError, match="overlap"):
        lm.attention8(big[:-1], *a[1:], out=big[1:])


@pytest.mark.parametrize("lens", [[300] * 3, [3000, 17, 0], [(9 * r) % 70 for r in range(900)]])
def test_repeated_replayed_and_on_another_stream(lens):
    """The same bits from every call: eager, on a side stream, and from graphs that are replayed in
    between (each with a workspace of its own)."""
    a = make(lens, 8, 2, 128, torch.bfloat16, torch.float8_e4m3fn, 16)
    want, wl = lm.attention8(*a)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out, lse = lm.attention8(*a, stream=side)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wl)
    graphs = []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            graphs[-1].got = lm.attention8(*a)
    for i in range(6):
        g = graphs[i % 2]
        g.got[0].fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(g.got[0], want) and torch.equal(g.got[1], wl)
        again, _ = lm.attention8(*a)
        assert torch.equal(again, want)


def test_a_cache_past_32_bits():
    """Pages whose codes lie more than 2^32 bytes behind the first one's."""
    pages, page, H, D = 66000, 256, 2, 128
    kc = torch.empty((pages, page, H, D), dtype=torch.int8, device="cuda")
    vc, ks = torch.empty_like(kc), torch.full((pages, H), 0.01, device="cuda")
    ids = [0, 65999, 40000, 33000]
    for c in (kc, vc):
        c[ids] = torch.randint(-127, 128, (4, page, H, D), dtype=torch.int8, device="cuda")
    tables = torch.tensor([ids, ids[::-1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([1024, 900], dtype=torch.int32, device="cuda")
    q = torch.randn((2, 4, D), device="cuda")
    out, lse = lm.attention8(q, kc, vc, ks, ks, tables, lens)
    small = torch.tensor([[0, 1, 2, 3], [3, 2, 1, 0]], dtype=torch.int32, device="cuda")
    want, wl = lm.attention8(q, kc[ids], vc[ids], ks[:4], ks[:4], small, lens)
    assert torch.equal(out, want) and torch.equal(lse, wl)


def test_refusals():
    q, kc, vc, ks, vs, tables, lens = make([40, 9], 4, 2, 64, torch.float16, torch.int8, 16)
    good = dict(q=q, k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs, tables=tables, lengths=lens)
    wide = torch.zeros((4, 16, 2, 72), dtype=torch.int8, device="cuda")
    for kw in (dict(q=q.double()), dict(q=q[:, :3]), dict(q=q[..., :48]), dict(k_cache=kc.half()),
               dict(v_cache=vc.view(torch.float8_e4m3fn)), dict(k_scale=ks.half()),
               dict(v_scale=vs[:, :1]), dict(lengths=lens.long()), dict(tables=tables[:1]),
               dict(window=-1), dict(max_len=-1), dict(out=q[:1].expand(2, 4, 64)),
               dict(q=q.clone().requires_grad_()), dict(k_cache=kc[..., :40], v_cache=vc[..., :40],
                                                        q=q[..., :40]),
               dict(k_cache=wide[:, :, :, 1:65], v_cache=wide[:, :, :, :64], k_scale=ks[:4],
                    v_scale=vs[:4])):
        with pytest.raises((ValueError, TypeError)):
            lm.attention8(**{**good, **kw})
    with torch.no_grad():
        lm.attention8(**{**good, "q": q.clone().requires_grad_()})
    out, lse = lm.attention8(q[:0], kc, vc, ks, vs, tables[:0], lens[:0])
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
