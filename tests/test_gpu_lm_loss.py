"""Token losses over a vocabulary and their gradients, against float64, against
differences of the loss, and through torch's autograd."""
import pytest
import torch

import lm_ref
from ctc_prefix_beam_amd import lm

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def make(N, V, H, dtype, bias=True, seed=0, pad=0.1):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((N, H), generator=g).to(dtype).cuda()
    w = (torch.randn((V, H), generator=g) * (3 / H ** 0.5)).to(dtype).cuda()
    b = torch.randn((V,), generator=g).cuda() if bias else None
    t = torch.randint(0, V, (N,), generator=g, dtype=torch.int32)
    t[torch.rand(N, generator=g) < pad] = -1
    grad = (torch.rand((N,), generator=g) * 2 - 1) * (1024.0 if dtype == torch.float16 else 1) / max(N, 1)
    return x, w, t.cuda(), b, grad.cuda()


def check(x, w, t, b, grad):
    loss, lse = lm.token_loss_forward(x, w, t, b)
    dx, dw, db = lm.token_loss_backward(grad, x, w, t, lse, b)
    want, tol = lm_ref.loss(x, w, t, b, grad)
    for name, got, a, e in zip(("loss", "lse", "dx", "dw", "dbias"), (loss, lse, dx, dw, db), want,
                               tol):
        if got is None:
            assert name == "dbias" and b is None
            continue
        off = (got.cpu().double() - a).abs() - e
        assert torch.isfinite(got).all() and (off <= 0).all(), (name, float(off.max()))
    assert dx.dtype == x.dtype and dw.dtype == w.dtype and loss.dtype == torch.float32
    return loss, lse, dx, dw, db


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,V,H", [
    (1, 2, 8), (1, 5000, 512), (3, 29, 64), (16, 512, 40), (17, 130, 72), (33, 1024, 256),
    (64, 257, 128), (129, 1000, 192), (300, 5000, 64), (257, 640, 1024), (1000, 129, 136)])
def test_sizes(dtype, N, V, H):
    check(*make(N, V, H, dtype, bias=N % 2 == 1, seed=N + V))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H", [1, 3, 7, 9, 63, 65, 127, 250])
def test_odd_hidden(dtype, H):
    check(*make(70, 300, H, dtype, seed=H))


@pytest.mark.parametrize("dtype", TYPES)
def test_strided_rows(dtype):
    x, w, t, b, grad = make(50, 200, 64, dtype)
    want = check(x, w, t, b, grad)
    for extra, first in ((8, 0), (8, 8), (5, 0), (8, 3)):   # aligned rows and others
        xs = torch.full((50, 64 + extra + first), float("nan"), dtype=dtype, device="cuda")
        ws = torch.full((200, 64 + extra + first), float("nan"), dtype=dtype, device="cuda")
        xs[:, first:first + 64], ws[:, first:first + 64] = x, w
        got = check(xs[:, first:first + 64], ws[:, first:first + 64], t, b, grad)
        assert all(torch.equal(a, c) for a, c in zip(got, want))


@pytest.mark.parametrize("dtype", TYPES)
def test_targets_outside_the_vocabulary_have_no_part(dtype):
    x, w, t, b, grad = make(40, 100, 64, dtype, pad=0.0)
    t[3], t[7], t[20], t[39] = -1, 100, 2 ** 31 - 1, -2 ** 31
    loss, lse, dx, dw, db = check(x, w, t, b, grad)
    out = [3, 7, 20, 39]
    assert (loss[out] == 0).all() and (dx[out] == 0).all()
    grad2 = grad.clone()
    grad2[out] = float("nan")
    _, dw2, db2 = lm.token_loss_backward(grad2, x, w, t, lse, b)
    assert torch.equal(dw2, dw) and torch.equal(db2, db)
    t[:] = -1
    loss, lse = lm.token_loss_forward(x, w, t, b)
    got = lm.token_loss_backward(grad, x, w, t, lse, b)
    assert not loss.any() and not any(a.any() for a in got)


@pytest.mark.parametrize("dtype", TYPES)
def test_masked_vocabulary_and_large_logits(dtype):
    x, w, t, b, grad = make(60, 300, 64, dtype, bias=True)
    t.clamp_(min=0, max=150)
    b[200:] = float("-inf")                # labels that may not be emitted
    loss, lse = lm.token_loss_forward(x, w, t, b)
    want, tol = lm_ref.loss(x, w[:200], t, b[:200], grad)
    assert ((loss.cpu().double() - want[0]).abs() <= tol[0]).all()
    dx, dw, db = lm.token_loss_backward(grad, x, w, t, lse, b)
    assert torch.isfinite(dx).all() and not dw[200:].any() and not db[200:].any()
    # the type's lowest value as a mask, and logits in the hundreds
    b[200:] = torch.finfo(torch.float32).min
    other = lm.token_loss_forward(x, w, t, b)
    assert torch.equal(other[0], loss) and torch.equal(other[1], lse)
    check(x, w * 30, t, None, grad)


def test_row_without_a_finite_logit():
    x, w, t, b, grad = make(4, 50, 16, torch.float32)
    b[:] = float("-inf")
    loss, lse = lm.token_loss_forward(x, w, t, b)
    assert (lse == float("-inf")).all()


def test_f16_gradients_keep_small_and_large_rows():
    """Row weights far apart and far from 1: d stays in f16's range."""
    for size in (1e-6, 1.0, 1e4):
        x, w, t, b, grad = make(64, 200, 64, torch.float16)
        x = x * 0.1
        loss, lse = lm.token_loss_forward(x, w, t, b)
        dx, dw, db = lm.token_loss_backward(grad * size, x, w, t, lse, b)
        want, tol = lm_ref.loss(x, w, t, b, grad * size)
        for got, a, e in zip((dx, dw, db), want[2:], tol[2:]):
            fits = a.abs() < 60000
            off = (got.cpu().double() - a).abs() - e
            assert (off[fits] <= 0).all()


@pytest.mark.parametrize("N,V,H", [(3, 319, 1377), (1, 700, 2048), (40, 200, 2000),
                                   (300, 128, 4096)])
def test_f32_products_over_long_rows(N, V, H):
    """Their 2-norms, to what sums in parts allow.  The logits reach 16, whose float32
    are 2^-20 apart, and a rounding is 0.29 of that at the root mean square: H / 128
    additions of parts and the rounding of lse lose 0.29 2^-20 (sqrt(H / 128) + 1),
    additions within the parts, of sqrt(128 / H) the size, the same times sqrt(H / 128)
    sqrt(128) sqrt(128 / H) / 3.  Twice their sum is allowed."""
    x, w, t, b, grad = make(N, V, H, torch.float32, seed=H, pad=0)
    _, lse = lm.token_loss_forward(x, w, t, b)
    got = lm.token_loss_backward(grad, x, w, t, lse, b)
    want, _ = lm_ref.loss(x, w, t, b, grad)
    tol = 2 * 0.29 * 2.0 ** -20 * ((H / 128) ** 0.5 + 1 + 128 ** 0.5 / 3)
    for name, a, e in zip(("dx", "dw", "dbias"), got, want[2:]):
        assert (a.cpu().double() - e).norm() <= tol * e.norm(), name


@pytest.mark.parametrize("bias", [True, False])
def test_gradient_against_differences(bias):
    x, w, t, b, grad = make(24, 60, 32, torch.float32, bias=bias, seed=5)
    _, lse = lm.token_loss_forward(x, w, t, b)
    got = lm.token_loss_backward(grad, x, w, t, lse, b)
    g = torch.Generator().manual_seed(1)
    ins = [x, w] + ([b] if bias else [])

    def f(parts):
        l, _ = lm.token_loss_forward(parts[0], parts[1], t, parts[2] if bias else None)
        return (l.double() * grad.double()).sum()
    for i, a in enumerate(ins):
        way = torch.randn(a.shape, generator=g).cuda()
        h = 2.0 ** -7
        up, down = list(ins), list(ins)
        up[i], down[i] = a + h * way, a - h * way
        diff = (f(up) - f(down)) / (2 * h)
        want = (got[i].double() * way.double()).sum()
        # h^2 / 6 of the third derivative along `way`, and float32 losses over 2h
        size = (grad.abs().double().sum() + 1) * float(way.double().norm()) ** 2
        assert abs(float(diff - want)) <= h * h * float(size) + 2.0 ** -20 * 20 / h


def test_autograd_matches_the_functions_and_needs_only_what_is_asked():
    x, w, t, b, grad = make(30, 90, 48, torch.bfloat16)
    _, lse = lm.token_loss_forward(x, w, t, b)
    want = lm.token_loss_backward(grad, x, w, t, lse, b)
    xs, ws, bs = (a.clone().requires_grad_() for a in (x, w, b))
    (lm.token_loss(xs, ws, t, bs) * grad).sum().backward()
    assert all(torch.equal(a.grad, c) for a, c in zip((xs, ws, bs), want))
    ws = w.clone().requires_grad_()
    (lm.token_loss(x, ws, t) * grad).sum().backward()
    assert ws.grad is not None
    only = lm.token_loss_backward(grad, x, w, t, lse, b, need=(True, False, False))
    assert torch.equal(only[0], want[0]) and only[1] is None and only[2] is None


@pytest.mark.parametrize("N,V", [(70000, 5003), (70000, 9001)])
def test_several_pieces_of_the_vocabulary(N, V):
    """Enough rows that d is made in several pieces: dx is summed over them."""
    H = 64
    x, w, t, b, grad = make(N, V, H, torch.bfloat16, seed=9)
    loss, lse = lm.token_loss_forward(x, w, t, b)
    dx, dw, db = lm.token_loss_backward(grad, x, w, t, lse, b)
    rows = torch.randperm(N, generator=torch.Generator().manual_seed(2))[:200].cuda()
    want, tol = lm_ref.loss(x[rows], w, t[rows], b, grad[rows])
    assert ((loss[rows].cpu().double() - want[0]).abs() <= tol[0]).all()
    assert ((dx[rows].cpu().double() - want[2]).abs() <= tol[2]).all()
    # dw and dbias of all rows in float64 on the GPU
    z = x.double() @ w.double().t() + b.double()
    ok = t >= 0
    d = torch.softmax(z, 1)
    d[torch.nonzero(ok)[:, 0], t[ok].long()] -= 1
    d *= torch.where(ok, grad, 0.0).double()[:, None]
    dw64 = d.t().contiguous() @ x.double()
    off = (dw.double() - dw64).norm() / dw64.norm()
    assert float(off) < 2 ** -8      # two roundings to bf16, each about 2^-9.2 in the mean square
    db64 = d.sum(0)
    assert float((db.double() - db64).norm() / db64.norm()) < 2 ** -16


def test_no_rows():
    x, w, t, b, grad = make(5, 90, 48, torch.bfloat16)
    loss, lse = lm.token_loss_forward(x[:0], w, t[:0], b)
    assert loss.shape == (0,) and lse.shape == (0,)
    dx, dw, db = lm.token_loss_backward(grad[:0], x[:0], w, t[:0], lse, b)
    assert dx.shape == (0, 48) and not dw.any() and not db.any()


def test_repeats_give_the_same_bits_on_another_stream_and_in_a_graph():
    x, w, t, b, grad = make(200, 3000, 128, torch.float16)

    def f(stream=None):
        loss, lse = lm.token_loss_forward(x, w, t, b, stream=stream)
        return (loss, lse) + lm.token_loss_backward(grad, x, w, t, lse, b, stream=stream)
    want = [a.clone() for a in f()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = f(side)
    side.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = f()
    for i in range(4):
        for a in out:
            a.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(out, want)), i
        torch.ones(1000, device="cuda").cumsum(0)


def test_refusals():
    x, w, t, b, grad = make(5, 90, 48, torch.bfloat16)
    _, lse = lm.token_loss_forward(x, w, t, b)
    bad = [
        ("w must be", (x, w[:, :40], t, b)), ("w must be", (x, w.float(), t, b)),
        ("targets", (x, w, t.long(), b)), ("targets", (x, w, t[:4], b)),
        ("bias", (x, w, t, b.bfloat16())), ("bias", (x, w, t, b[:9])),
        ("x must be", (x.t(), w, t, b)), ("bfloat16", (x.double(), w.double(), t, b)),
        ("GPU", (x.cpu(), w, t, b)), ("targets", (x, w, t.cpu(), b))]
    for match, args in bad:
        with pytest.raises(ValueError, match=match):
            lm.token_loss_forward(*args)
    with pytest.raises(ValueError, match="grad"):
        lm.token_loss_backward(grad.double(), x, w, t, lse, b)
    with pytest.raises(ValueError, match="lse"):
        lm.token_loss_backward(grad, x, w, t, lse[:2], b)
    with pytest.raises(ValueError, match="vocab"):
        lm.token_loss_forward(x, w[:0], t, None)
