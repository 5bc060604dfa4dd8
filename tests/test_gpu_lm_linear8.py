"""Rows as 8-bit codes, and the products of such rows, against 64 bits."""
import math

import pytest
import torch

import lm_ref8
from ctc_prefix_beam_amd import lm

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def rows(N, H, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((N, H), generator=g) * torch.exp2(torch.randint(-5, 6, (N, 1), generator=g))
    return x.to(dtype).cuda()


def weight(M, H, seed=1):
    """Codes of every kind, -128 too, in rows that end where they end, and scales."""
    g = torch.Generator().manual_seed(seed)
    w = torch.randint(-128, 128, (M, H), generator=g, dtype=torch.int32).to(torch.int8)
    return w.cuda(), (torch.rand(M, generator=g) + 0.5).cuda() / 4000


def check(x, w, ws, bias=None, **kw):
    out = lm.linear8(x, w, ws, bias, **kw)
    codes, scales = lm_ref8.quantize(x)
    want, tol = lm_ref8.linear(codes, scales, w, ws, bias, x.dtype)
    assert out.dtype == x.dtype
    assert ((out.cpu().double() - want).abs() <= tol).all(), float(
        ((out.cpu().double() - want).abs() / tol).max())
    return out


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H", [1, 3, 16, 100, 387, 512, 2048, 4096, 5003, 17000, 40008])
def test_codes_and_scales(dtype, H):
    for N in (1, 70, 1100) if H < 6000 else (3,):
        x = rows(N, H, dtype, H)
        codes, scales = lm.quantize_rows(x)
        want, s = lm_ref8.quantize(x)
        assert torch.equal(scales.cpu(), s)
        assert torch.equal(codes.cpu().double(), want)
        assert codes.stride(0) % 16 == 0
        whole = codes.as_strided((N, codes.stride(0)), (codes.stride(0), 1))
        assert (whole[:, H:] == 0).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H", [5, 8, 387, 512, 2047, 4100])
def test_rows_that_begin_anywhere(dtype, H):
    """Values and codes at addresses that are multiples of their own size only, a wave or a
    workgroup to each row, and nothing written beside the rows."""
    for N in (9, 1030):
        big = rows(N, H + 9, dtype, H)
        for at in range(4 if N < 100 else 2):
            x = big[:, at:at + H]
            want, s = lm_ref8.quantize(x)
            codes, scales = lm.quantize_rows(x)
            assert torch.equal(scales.cpu(), s) and torch.equal(codes.cpu().double(), want)
            for step in (H, H + 3):
                space = torch.full((N * step + 32,), 99, dtype=torch.int8, device="cuda")
                part = space[16 + at:]
                lm._check(lm.lib().ctcpb_lm_quantize_rows(lm._pack(
                    lm._QUANTIZE, x.data_ptr(), part.data_ptr(), scales.data_ptr(), x.stride(0),
                    step, lm._TYPES[dtype], N, H), torch.cuda.current_stream().cuda_stream))
                got = part[:N * step].view(N, step)
                assert torch.equal(got[:, :H].cpu().double(), want)
                assert (got[:, H:min(step, -(-H // 16) * 16)] == 0).all()
                assert (space[:16 + at] == 99).all() and (part[N * step:] == 99).all()


def test_more_rows_than_one_launch_takes():
    N = (1 << 22) + 70
    x = rows(100, 9, torch.float16).repeat(N // 100 + 1, 1)[:N]
    codes, scales = lm.quantize_rows(x)
    want, s = lm_ref8.quantize(x[:100])
    for a in (0, (1 << 22) - 300, N - 300):
        at = a // 100 * 100
        assert torch.equal(codes[at:at + 100].cpu().double(), want)
        assert torch.equal(scales[at:at + 100].cpu(), s)
    assert torch.equal(codes, codes[:100].repeat(N // 100 + 1, 1)[:N])
    assert torch.equal(scales, scales[:100].repeat(N // 100 + 1)[:N])


@pytest.mark.parametrize("dtype", TYPES)
def test_quotients_next_to_a_half(dtype):
    """Every value is n + 1/2 steps, or a neighbour of that in the type: halves go to the even
    code, the others to their own side."""
    g = torch.Generator().manual_seed(0)
    N, H = 200, 256
    most = (torch.rand((N, 1), generator=g) + 0.5).to(dtype)
    step = most.float() / 127
    n = torch.arange(H - 1).float() % 127 + 0.5
    x = (n * step).to(dtype)
    off = torch.randint(-1, 2, x.shape, generator=g)
    up, down = torch.nextafter(x, x * 2), torch.nextafter(x, x * 0)
    x = torch.where(off > 0, up, torch.where(off < 0, down, x)).clamp(max=most)
    x = torch.cat((x, most), 1)
    x = torch.cat((x, -x, x), 0)
    x[2 * N:, :-1] = (n / 127).to(dtype)       # a scale of 1/127 of one
    x[2 * N:, -1] = 1
    extra = torch.cat((torch.arange(-127, 127).float() + 0.5, torch.tensor([127.0, 0.0])))
    x = torch.cat((x, extra.to(dtype)[None], extra.to(dtype)[None] * 2.0 ** -3)).cuda()
    codes, scales = lm.quantize_rows(x)
    want, s = lm_ref8.quantize(x)
    assert torch.equal(scales.cpu(), s) and torch.equal(codes.cpu().double(), want)
    assert want[-1, :4].tolist() == [-126, -126, -124, -124]   # exact halves: a scale of 1/8


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_at_the_ends_of_the_type(dtype):
    info = torch.finfo(dtype)
    x = torch.zeros((9, 24), dtype=dtype)
    x[1, 3], x[1, 4] = info.max, -info.max
    x[2] = torch.arange(24).to(dtype) * info.smallest_normal
    x[3] = torch.arange(24).to(dtype) * (info.smallest_normal * 2.0 ** -6)
    x[4, 5], x[5, 6], x[6, 7] = math.nan, math.inf, -math.inf
    x[4, 0] = 3.0
    x[7] = -0.0
    x[8] = torch.arange(24).to(dtype) - 12
    codes, scales = lm.quantize_rows(x.cuda())
    want, s = lm_ref8.quantize(x)
    assert torch.equal(scales.cpu().nan_to_num(-1), s.nan_to_num(-1))
    assert torch.equal(codes.cpu().double(), want)
    w, ws = weight(33, 24)
    out = lm.linear8(x.cuda(), w, ws)
    bad = torch.isnan(s)
    assert bad.tolist() == [False] * 4 + [True] * 3 + [False] * 2
    assert torch.isnan(out.cpu()[bad]).all()
    if dtype != torch.float16:
        assert torch.isfinite(out.cpu()[~bad]).all()
    assert (out[0] == 0).all() and (out[7] == 0).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,M,H", [
    (1, 1, 1), (1, 29, 64), (1, 5000, 512), (3, 319, 1377), (5, 7, 16), (16, 64, 128), (17, 65, 130),
    (32, 5000, 512), (33, 1000, 2048), (64, 128, 8192), (65, 35, 64), (100, 256, 4096),
    (255, 257, 259), (256, 512, 512), (875, 1531, 387), (1000, 100, 1000), (2000, 2000, 600)])
def test_sizes(dtype, N, M, H):
    x = rows(N, H, dtype, N)
    w, ws = weight(M, H)
    g = torch.Generator().manual_seed(2)
    bias = torch.randn(M, generator=g).cuda()
    check(x, w, ws)
    check(x, w, ws, bias)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,M,H", [
    (1, 1, 1), (1, 100, 32768), (1, 50000, 40), (2, 77, 16000), (4, 129, 8192), (5, 33, 5003),
    (16, 20000, 64), (16, 48, 2048), (17, 1000, 100), (31, 333, 1000), (32, 5000, 512),
    (32, 65, 1024), (32, 65, 1025),
    (32, 4100, 4000), (31, 60, 4096), (32, 60, 4096), (3, 60, 42000), (32, 4111, 2048), (20, 50, 6553), (3, 300, 43000)])
def test_few_rows(dtype, N, M, H):
    """Rows on both sides of what one launch does, with weights in rows that can be read past
    their ends, where anything may lie; as values and as codes."""
    x = rows(N, H, dtype, N)
    w, ws = weight(M, H)
    wide = torch.full((M, -(-H // 16) * 16 + 16), 99, dtype=torch.int8, device="cuda")[:, :H]
    wide.copy_(w)
    bias = torch.randn(M).cuda()
    want = check(x, w, ws, bias)
    assert torch.equal(check(x, wide, ws, bias), want)
    codes, s = lm.quantize_rows(x)
    assert torch.equal(lm.linear8(codes, wide, ws, bias, x_scale=s, dtype=dtype), want)
    apart = torch.zeros((N, H + 3), dtype=dtype, device="cuda")[:, 1:H + 1]
    apart.copy_(x)
    assert torch.equal(lm.linear8(apart, wide, ws, bias), want)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,M,H", [
    (1, 77, 16000), (1, 29, 16384), (2, 40, 8192), (3, 65, 5001), (4, 5000, 1100), (5, 65, 3200),
    (7, 33, 2300), (8, 20, 2048), (9, 40, 1800), (13, 33, 1250), (16, 70, 1024), (17, 40, 960)])
def test_few_long_rows(dtype, N, M, H):
    """Rows that several waves quantise, with one of zeros, one of a single value and one that is
    not finite among them."""
    x = rows(N, H, dtype, N)
    if N > 3:
        x[0], x[1, 1:] = 0, 0
        x[3, H - 1] = math.inf
    w, ws = weight(M, -(-H // 16) * 16)
    w = w[:, :H]
    out = lm.linear8(x, w, ws)
    codes, s = lm_ref8.quantize(x)
    if N > 3:
        assert torch.isnan(out[3]).all() and (out[0] == 0).all()
        codes, s, x, out = (t[torch.arange(N) != 3] for t in (codes, s, x, out.cpu()))
    want, tol = lm_ref8.linear(codes, s, w, ws, None, dtype)
    assert ((out.cpu().double() - want).abs() <= tol).all()


@pytest.mark.parametrize("N,M,H", [(1, 40, 131071), (3, 70, 100000), (300, 40, 65536)])
def test_long_sums_stay_whole(N, M, H):
    """Sums of up to 2^31 - 128^2, exact in 32 bits."""
    x = torch.full((N, H), 2.5, device="cuda")
    w = torch.full((M, H), -128, dtype=torch.int8, device="cuda")
    one = torch.ones(M, device="cuda")
    out = lm.linear8(x, w, one)
    want = -128.0 * 127 * H * float(torch.tensor(2.5) / 127)
    assert ((out.double() - want).abs() <= 2.0 ** -22 * abs(want)).all()
    xs = torch.ones(N, device="cuda")
    out = lm.linear8(w[:1].expand(N, H), w, one, x_scale=xs, dtype=torch.float32)
    assert (out.double() == 128.0 * 128 * H).all() or H % 2   # (131071: 2^31 - 2^14, 17 bits)
    assert ((out.double() - 128.0 * 128 * H).abs() <= 2.0 ** -23 * 128.0 * 128 * H).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_a_row_is_the_same_among_others(dtype):
    """Whatever kernels the number of rows takes: sums are exact, and what follows is alike."""
    M, H = 777, 1032
    x = rows(2500, H, dtype)
    w, ws = lm.quantize_rows(torch.randn(M, H, device="cuda"))
    bias = torch.randn(M, device="cuda")
    want = lm.linear8(x, w, ws, bias)
    for n in (1, 5, 16, 17, 31, 40, 100, 300, 1100):
        assert torch.equal(lm.linear8(x[7:7 + n], w, ws, bias), want[7:7 + n]), n
        some = lm.linear8(x[7:7 + n], w[:500], ws[:500], bias[:500])
        assert torch.equal(some, want[7:7 + n, :500]), n


def test_large_tiles_against_products_in_pieces():
    """Sizes that fill the card with the largest tiles, with ends that do not, against exact
    float64 products on the GPU."""
    for N, M, H in ((8192, 8192, 512), (20000, 1000, 1024), (4097, 5003, 640)):
        x = rows(N, H, torch.bfloat16)
        w, ws = weight(M, H)
        out = lm.linear8(x, w, ws)
        codes, s = lm.quantize_rows(x)
        for a in range(0, N, 4096):
            y = torch.mm(codes[a:a + 4096].double(), w.double().t())
            y *= s[a:a + 4096].double()[:, None] * ws.double()
            assert ((out[a:a + 4096].double() - y).abs() <= (2.0 ** -8 + 2.0 ** -21) * y.abs()).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_codes_as_input(dtype):
    x = rows(70, 130, torch.float32)
    codes, s = lm.quantize_rows(x)
    w, ws = weight(45, 130)
    bias = torch.randn(45).cuda()
    out = lm.linear8(codes, w, ws, bias, x_scale=s, dtype=dtype)
    assert out.dtype == dtype
    assert torch.equal(out, lm.linear8(codes.contiguous(), w, ws, bias, x_scale=s, dtype=dtype))
    assert torch.equal(out.float() if dtype == torch.float32 else out,
                       lm.linear8(x, w, ws, bias).to(dtype))
    assert lm.linear8(codes, w, ws, x_scale=s).dtype == torch.bfloat16
    # parts of wider rows, whose other codes have no part in the sums
    wide = [torch.full((n, 160), 77, dtype=torch.int8, device="cuda") for n in (70, 45)]
    for t, c in zip(wide, (codes, w)):
        t[:, :130] = c
    got = lm.linear8(wide[0][:, :130], wide[1][:, :130], ws, bias, x_scale=s, dtype=dtype)
    assert torch.equal(got, out)
    assert torch.equal(lm.linear8(x, wide[1][:, :130], ws, bias), lm.linear8(x, w, ws, bias))


def test_strides():
    """Rows of x, w, out that lie apart, begin anywhere and end at the end of their memory."""
    g = torch.Generator().manual_seed(0)
    big = torch.randn((40, 333), generator=g).cuda()
    w, ws = weight(50, 300)
    wide = torch.zeros((50, 320), dtype=torch.int8, device="cuda")
    for at in (0, 1, 16, 20):
        x = big[::2, at + 1:at + 301]
        part = wide[:, at:at + 300]
        part.copy_(w)
        space = torch.full((20, 64), 9.0, device="cuda")
        out = lm.linear8(x, part, ws, out=space[:, 3:53])
        assert torch.equal(out, check(x.contiguous(), w, ws))
        assert (space[:, :3] == 9).all() and (space[:, 53:] == 9).all()
        half = torch.full((20, 56), 9.0, dtype=torch.float16, device="cuda")
        got = lm.linear8(x.half(), part, ws, out=half[:, :50])
        assert torch.equal(got, check(x.half(), w, ws)) and (half[:, 50:] == 9).all()
    one = big[:1, :300].expand(5, 300)   # read, rows may share their memory
    assert torch.equal(lm.linear8(one, w, ws)[4:], check(one.contiguous(), w, ws)[:1])


def test_graphs_streams_and_no_rows():
    x = rows(300, 2048, torch.bfloat16)
    w, ws = weight(200, 2048)
    want = check(x, w, ws)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = lm.linear8(x, w, ws, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = lm.linear8(x, w, ws)
        codes, s = lm.quantize_rows(x)
    for i in range(4):
        got.zero_()
        codes.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        again, t = lm.quantize_rows(x)
        assert torch.equal(again, codes) and torch.equal(s, t)
    assert lm.linear8(x[:0], w, ws).shape == (0, 200)
    codes, s = lm.quantize_rows(x[:0])
    assert codes.shape == (0, 2048) and s.shape == (0,)


def test_refusals():
    x = rows(4, 32, torch.float16)
    w, ws = weight(8, 32)
    codes, s = lm.quantize_rows(x)
    good = dict(x=x, w=w, w_scale=ws)
    for kw in (dict(x=x.double()), dict(x=x[:, :31]), dict(x=x[0]), dict(x=x.t()), dict(w=w.short()),
               dict(w=w.t()), dict(w_scale=ws[:7]), dict(w_scale=ws.half()), dict(bias=ws.half()),
               dict(bias=ws[:3]), dict(x=codes), dict(x_scale=s), dict(x=codes, x_scale=s[:2]),
               dict(dtype=torch.float32), dict(x=codes, x_scale=s, dtype=torch.int8),
               dict(out=torch.zeros((4, 8), device="cuda")),
               dict(out=torch.zeros((1, 8), dtype=x.dtype, device="cuda").expand(4, 8)),
               dict(out=torch.zeros((8, 4), dtype=x.dtype, device="cuda").t()),
               dict(x=x.clone().requires_grad_()), dict(w=w[:, :0], x=x[:, :0]), dict(w=w.cpu()),
               dict(w=w[:0], w_scale=ws[:0])):
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            lm.linear8(**{**good, **kw})
    with pytest.raises(RuntimeError, match="131071"):
        lm.linear8(torch.zeros((1, 131072), device="cuda"),
                   torch.zeros((1, 131072), dtype=torch.int8, device="cuda"), ws[:1])
    for bad in (x.double(), x[0], x[:, :0], x.t(), codes, x.clone().requires_grad_()):
        with pytest.raises(ValueError):
            lm.quantize_rows(bad)


def test_out_does_not_overlap_its_inputs():
    x = rows(40, 64, torch.float16)
    w, ws = weight(64, 64)
    want = lm.linear8(x, w, ws)
    for bad in (x, x.as_strided((40, 64), (32, 1))):
        with pytest.raises(ValueError, match="overlap"):
            lm.linear8(x, w, ws, out=bad)
    one = torch.empty((8192,), dtype=torch.uint8, device="cuda")
    part = one[:4096].view(torch.int8).view(64, 64)
    part.copy_(w)
    with pytest.raises(ValueError, match="overlap"):
        lm.linear8(x, part, ws, out=one[2048:2048 + 5120].view(torch.float16).view(40, 64))
    # the halves of one matrix
    both = torch.zeros((40, 128), dtype=torch.float16, device="cuda")
    for a, b in ((0, 64), (64, 0)):
        both[:, a:a + 64] = x
        lm.linear8(both[:, a:a + 64], w, ws, out=both[:, b:b + 64])
        assert torch.equal(both[:, b:b + 64], want) and torch.equal(both[:, a:a + 64], x)
    with pytest.raises(ValueError, match="overlap"):
        lm.linear8(both[:, :64], w, ws, out=both[:, 63:127])
    with pytest.raises(ValueError, match="overlap"):
        lm.linear8(both[:, 64:], w, ws, out=both[:, 1:65])
