"""Attention of one token per request over the paged cache, against float64."""
import math

import pytest
import torch

import lm_ref
from ctc_prefix_beam_amd import lm

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def make(lengths, Hq, Hkv, D, dtype, page, order="thd", seed=0, spare=1, width=None, nan=True):
    """q, caches, tables, lengths; every slot no request owns holds NaN."""
    g = torch.Generator().manual_seed(seed)
    lens = torch.tensor(lengths, dtype=torch.int32)
    have = [-(-max(n, 0) // page) for n in lengths]
    pages = sum(have) + spare
    shape = (pages, page, Hkv, D) if order == "thd" else (pages, Hkv, page, D)
    kc, vc = torch.randn(shape, generator=g), torch.randn(shape, generator=g)
    if order == "htd":
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
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
    if nan:
        kc[~used], vc[~used] = math.nan, math.nan
    q = 2 * torch.randn((len(lengths), Hq, D), generator=g)
    kc, vc = kc.to(dtype), vc.to(dtype)
    return tuple(x.cuda() for x in (q.to(dtype), kc, vc, tables, lens))


def check(q, kc, vc, tables, lens, page, scale=None, window=0, **kw):
    out, lse = lm.attention(q, kc, vc, tables, lens, scale=scale, window=window, **kw)
    s = q.shape[2] ** -0.5 if scale is None else scale
    wo, wl, to, tl = lm_ref.attention(q, kc, vc, tables, lens, s, window, page)
    out, lse = out.cpu().double(), lse.cpu().double()
    assert torch.isfinite(out).all()
    assert ((out - wo).abs() <= to).all(), float(((out - wo).abs() - to).max())
    dead = wl == -math.inf
    assert torch.equal(lse == -math.inf, dead)
    assert ((lse - wl).abs()[~dead] <= tl[~dead]).all()
    return out


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [8, 40, 64, 72, 80, 96, 128, 136, 192, 256])
def test_head_dims(dtype, D):
    a = make([0, 1, 31, 32, 33, 150], 4, 2, D, dtype, 16, seed=D)
    check(*a, 16)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (5, 1), (8, 1), (16, 1), (17, 1), (40, 2),
                                    (64, 2), (12, 4)])
def test_head_groups(dtype, Hq, Hkv):
    check(*make([1, 0, 70, 300], Hq, Hkv, 64, dtype, 16, seed=Hq), 16)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("page", [4, 8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("order", ["thd", "htd"])
def test_pages_and_orders(dtype, page, order):
    check(*make([1, 3, 4, 5, 127, 128, 129, 513, 0, 1000], 6, 3, 64, dtype, page, order, page),
          page)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [1, 128, 257, 4096, 20011])
def test_one_request_split_over_its_length(dtype, n):
    check(*make([n], 8, 2, 128, dtype, 16, seed=n), 16)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("window", [1, 2, 15, 33, 200, 5000])
def test_window(dtype, window):
    check(*make([0, 1, 30, 64, 333, 4000], 4, 2, 64, dtype, 8, seed=window), 8, window=window)


def test_many_rows():
    lens = [(7 * r) % 90 for r in range(1500)]
    check(*make(lens, 4, 2, 64, torch.bfloat16, 16), 16)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [40, 64, 128, 256])
@pytest.mark.parametrize("width", [70, 140, 2000])
@pytest.mark.parametrize("window", [0, 37, 600])
def test_short_rows_in_tables_of_any_width(dtype, D, width, window):
    """What the lengths may be decides how the work is split, not what they are."""
    a = make([0, 1, 3, 16, 17, 0, 500, 64, 1100, 255], 6, 3, D, dtype, 16, seed=D, width=width)
    check(*a, 16, window=window)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Hq,Hkv,D", [(2, 1, 64), (20, 1, 64), (4, 2, 136)])
def test_many_rows_with_a_window(dtype, Hq, Hkv, D):
    lens = [(11 * r) % 70 for r in range(1100)]
    check(*make(lens, Hq, Hkv, D, dtype, 8, seed=D), 8, window=21)


def test_max_len_bounds_the_launch_not_the_result():
    a = make([5, 300, 77], 4, 2, 64, torch.bfloat16, 16, width=400)
    x = check(*a, 16)
    y = check(*a, 16, max_len=300)
    assert torch.allclose(x, y, rtol=2 ** -7, atol=2 ** -9)
    # lengths above the bound are clamped to it
    short = a[:4] + (a[4].clamp(max=128),)
    o, l = lm.attention(*a, max_len=128)
    p, m = lm.attention(*short, max_len=128)
    assert torch.equal(o, p) and torch.equal(l, m)


def test_strided_q_and_out():
    q, kc, vc, tables, lens = make([40, 9], 4, 2, 64, torch.float16, 16)
    fused = torch.zeros((2, 8, 65), dtype=q.dtype, device="cuda")
    fused[:, 2:6, 1:] = q
    big = torch.full((2, 9, 70), 3.0, dtype=q.dtype, device="cuda")
    want, _ = lm.attention(q, kc, vc, tables, lens)
    got, _ = lm.attention(fused[:, 2:6, 1:], kc, vc, tables, lens, out=big[:, 1:5, 3:67])
    assert torch.equal(got, want)
    assert (big[:, 0] == 3).all() and (big[:, 5:] == 3).all() and (big[:, :, :3] == 3).all()


def test_extreme_scores():
    """Large scores, equal scores, and keys that make a whole row -inf."""
    q, kc, vc, tables, lens = make([200, 64, 50], 2, 1, 64, torch.float32, 16, nan=False)
    check(q * 300, kc, vc, tables, lens, 16)      # one token takes all
    check(q * 0, kc, vc, tables, lens, 16)        # all tokens alike
    q[1], q[2] = 1.0, 1.0
    pages = tables[1, :4].long()
    kc[pages] = -math.inf
    out, lse = lm.attention(q, kc, vc, tables, lens)
    assert (out[1] == 0).all() and (lse[1] == -math.inf).all()
    assert torch.isfinite(out[[0, 2]]).all()
    kc[pages[0], 3] = 1.0                         # one finite token among them
    out, lse = lm.attention(q, kc, vc, tables, lens)
    t = vc[pages[0], 3, 0]
    assert torch.allclose(out[1, 0], t, atol=1e-6) and torch.allclose(lse[1], torch.tensor(8.0).cuda())
    low = torch.finfo(torch.float32).min
    kc[pages] = 0.0
    kc[pages, :, :, 0] = low                      # scores of the type's lowest value
    q[1] = 0.0
    q[1, :, 0] = 1.0
    out, lse = lm.attention(q, kc, vc, tables, lens, scale=1.0)
    mean = vc[pages].reshape(64, 64).double().mean(0)
    assert torch.allclose(out[1, 0].double(), mean, atol=1e-5)


def test_cache_past_32_bits():
    pages, page, H, D = 40000, 64, 8, 256
    kc = torch.empty((pages, page, H, D), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    tables = torch.tensor([[pages - 1, 3, pages - 2]], dtype=torch.int32, device="cuda")
    for p in tables[0].tolist():
        kc[p].normal_()
        vc[p].normal_()
    q = torch.randn((1, H, D), device="cuda").bfloat16()
    lens = torch.tensor([150], dtype=torch.int32, device="cuda")
    got = lm.attention(q, kc, vc, tables, lens)
    small = tables[0].long()
    want = lm.attention(q, kc[small].clone(), vc[small].clone(),
                        torch.arange(3, dtype=torch.int32, device="cuda")[None], lens)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_no_rows_and_no_width():
    q, kc, vc, tables, lens = make([40, 9], 4, 2, 64, torch.float16, 16)
    out, lse = lm.attention(q[:0], kc, vc, tables[:0], lens[:0])
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    out, lse = lm.attention(q, kc, vc, tables[:, :0], lens)
    assert not out.any() and (lse == -math.inf).all()


def test_repeats_give_the_same_bits_on_another_stream_and_in_a_graph():
    a = make([3000, 0, 700, 5000], 16, 2, 128, torch.bfloat16, 16)
    want = [t.clone() for t in lm.attention(*a)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = lm.attention(*a, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = lm.attention(*a)
    for i in range(4):
        for t in out:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, want)), i
        torch.ones(1000, device="cuda").cumsum(0)


def test_plan_store_attend_token_by_token():
    """A cache filled by prompts, then grown one token at a time, against the
    same tokens attended densely."""
    g = torch.Generator().manual_seed(1)
    R, Hq, H, D, page = 3, 4, 2, 64, 8
    c = lm.PagedCache(R, 64, H, D, torch.float32, page)
    ks, vs = torch.randn((R, 40, H, D), generator=g), torch.randn((R, 40, H, D), generator=g)
    n = [5, 0, 17]
    for step in range(6):
        cnt = [5, 0, 17] if step == 0 else [1, 1, step % 2]
        total = sum(cnt)
        plan = c.append(torch.tensor(cnt, dtype=torch.int32, device="cuda"), total)
        rows = torch.repeat_interleave(torch.arange(R), torch.tensor(cnt))
        pos = plan.positions.cpu().long()
        c.store(ks[rows, pos].cuda(), vs[rows, pos].cuda(), plan.slots)
        if step:
            n = [a + b for a, b in zip(n, cnt)]
        assert c.lengths.tolist() == n
        q = torch.randn((R, Hq, D), generator=g)
        out, _ = c.attend(q.cuda())
        for r in range(R):
            for h in range(Hq):
                if n[r] == 0:
                    assert not out[r].any()
                    continue
                k, v = ks[r, :n[r], h // 2].double(), vs[r, :n[r], h // 2].double()
                p = torch.softmax((k @ q[r, h].double()) / 8, 0)
                assert torch.allclose(out[r, h].cpu().double(), p @ v, atol=1e-5)


def test_refusals():
    q, kc, vc, tables, lens = make([40, 9], 4, 2, 64, torch.float16, 16)
    with pytest.raises(ValueError, match="multiple of kv_heads"):
        lm.attention(q[:, :3], kc, vc, tables, lens)
    with pytest.raises(ValueError, match="heads of"):
        lm.attention(q[:, :, :32], kc, vc, tables, lens)
    with pytest.raises(ValueError, match="multiple of 8"):
        lm.attention(q[:, :, :20], kc[..., :20], vc[..., :20], tables, lens)
    with pytest.raises(ValueError, match="k_cache"):
        lm.attention(q.bfloat16(), kc, vc, tables, lens)
    with pytest.raises(ValueError, match="lengths"):
        lm.attention(q, kc, vc, tables, lens.long())
    with pytest.raises(ValueError, match="tables"):
        lm.attention(q, kc, vc, tables[:1], lens)
    with pytest.raises(ValueError, match="window"):
        lm.attention(q, kc, vc, tables, lens, window=-1)
    with pytest.raises(ValueError, match="16-byte"):
        big = torch.zeros((kc.numel() + 1,), dtype=kc.dtype, device="cuda")
        lm.attention(q, big[1:].view(kc.shape), vc, tables, lens)
    wide = torch.zeros((2, 16, 1, 264), dtype=q.dtype, device="cuda")
    with pytest.raises(RuntimeError, match="256"):
        lm.attention(wide[:, 0], wide, wide, tables, lens)
