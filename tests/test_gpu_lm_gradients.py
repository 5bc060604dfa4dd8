"""Gradients of the token loss: as torch hands them on, and in several pieces."""
import pytest
import torch

from ctc_prefix_beam_amd import lm

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def make(N, V, H, dtype, bias=True, seed=0, pad=0.1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((N, H), generator=g, device="cuda").to(dtype)
    w = (torch.randn((V, H), generator=g, device="cuda") * (3 / H ** 0.5)).to(dtype)
    b = torch.randn((V,), generator=g, device="cuda") if bias else None
    t = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    t[torch.rand(N, generator=g, device="cuda") < pad] = -1
    scale = (1024.0 if dtype == torch.float16 else 1.0) / max(N, 1)
    grad = (torch.rand((N,), generator=g, device="cuda") * 2 - 1) * scale
    return x, w, t, b, grad


@pytest.mark.parametrize("dtype", TYPES)
def test_second_derivatives_are_refused(dtype):
    x, w, t, b, _ = make(20, 90, 48, dtype)
    ins = [a.clone().requires_grad_() for a in (x, w, b)]
    want = torch.autograd.grad(lm.token_loss(ins[0], ins[1], t, ins[2]).sum(), ins)
    loss = lm.token_loss(ins[0], ins[1], t, ins[2]).sum()
    got = torch.autograd.grad(loss, ins, create_graph=True)
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    with pytest.raises(RuntimeError, match="twice"):
        (loss + sum(a.float().pow(2).sum() for a in got)).backward()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N", [40, 300])
@pytest.mark.parametrize("garbage", [float("nan"), float("inf")])
def test_rows_without_a_target_hold_anything(dtype, N, garbage):
    """Their x may be NaN or infinite: no part of it gets into dx and dbias."""
    x, w, t, b, grad = make(N, 500, 64, dtype, pad=0.2)
    dead = t < 0
    _, lse = lm.token_loss_forward(x, w, t, b)
    want = lm.token_loss_backward(grad, x, w, t, lse, b)
    x[dead] = garbage
    loss, lse = lm.token_loss_forward(x, w, t, b)
    dx, _, db = lm.token_loss_backward(grad, x, w, t, lse, b, need=(True, False, True))
    assert (loss[dead] == 0).all() and (dx[dead] == 0).all()
    assert torch.equal(dx, want[0]) and torch.equal(db, want[2])


def check_norms(x, w, t, b, grad, got, tol):
    """Gradients against 64 bits in the 2-norm, dx in blocks of rows."""
    dx, dw, db = got
    (N, H), V = x.shape, w.shape[0]
    w64, dw64 = w.double(), torch.zeros((V, H), dtype=torch.float64, device="cuda")
    db64 = torch.zeros(V, dtype=torch.float64, device="cuda")
    for a in range(0, N, 20000):
        xs, ts = x[a:a + 20000].double(), t[a:a + 20000]
        z = xs @ w64.t()
        if b is not None:
            z += b.double()
        d = torch.softmax(z, 1)
        live = torch.nonzero(ts >= 0)[:, 0]
        d[live, ts[live].long()] -= 1
        d *= torch.where(ts >= 0, grad[a:a + 20000], 0.0).double()[:, None]
        want = d @ w64
        assert float((dx[a:a + 20000].double() - want).norm() / want.norm()) < tol
        dw64 += d.t().contiguous() @ xs
        db64 += d.sum(0)
    assert float((dw.double() - dw64).norm() / dw64.norm()) < tol
    if b is not None:
        assert float((db.double() - db64).norm() / db64.norm()) < 2.0 ** -16


NORM = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -16}


@pytest.mark.parametrize("dtype,N,V", [(torch.float32, 70000, 5003), (torch.float16, 140000, 5003),
                                       (torch.bfloat16, 140000, 9001)])
def test_pieces_of_the_vocabulary(dtype, N, V):
    """More d than is made at a time (1 GiB): dx is summed over two or three pieces.  Two
    roundings to the type (f32: sums of float32, 2^-16 of them at most)."""
    x, w, t, b, grad = make(N, V, 64, dtype, seed=9)
    assert N * (-(-V // 256) * 256) * x.element_size() > 1 << 30
    _, lse = lm.token_loss_forward(x, w, t, b)
    got = lm.token_loss_backward(grad, x, w, t, lse, b)
    check_norms(x, w, t, b, grad, got, NORM[dtype])


@pytest.mark.parametrize("dtype,N,V,H", [
    (torch.float32, 2000, 9000, 1024), (torch.float32, 9000, 2000, 1024),
    (torch.bfloat16, 8192, 17000, 1024), (torch.float16, 17000, 4096, 2048),
    (torch.bfloat16, 300, 1000, 64), (torch.float32, 875, 1000, 72)])
def test_products_cut_along_k(dtype, N, V, H):
    """All of a result, or its last rows (dw: of the vocabulary, dx: of the tokens), as a sum
    of parts of k.  Roundings as above."""
    x, w, t, b, grad = make(N, V, H, dtype, bias=False, seed=N)
    _, lse = lm.token_loss_forward(x, w, t, b)
    got = lm.token_loss_backward(grad, x, w, t, lse, b)
    check_norms(x, w, t, b, grad, got, NORM[dtype])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N,V,H", [(65, 700, 64), (300, 5000, 128), (4096, 3001, 257),
                                   (5000, 9000, 1024)])
def test_gradients_by_a_split_d_are_off_by_their_own_rounding(dtype, N, V, H):
    """d as two values is off by 2^-17 of itself (f16: 2^-22), a 256th of what the results
    lose in their own rounding; 2 % are allowed for it and the float32 sums."""
    x, w, t, b, grad = make(N, V, H, dtype, seed=N)
    xs, ws, bs = (a.clone().requires_grad_() for a in (x, w, b))
    (lm.token_loss(xs, ws, t, bs, split_d=True) * grad).sum().backward()
    z = torch.softmax(x.double() @ w.double().t() + b.double(), 1)
    live = torch.nonzero(t >= 0)[:, 0]
    z[live, t[live].long()] -= 1
    z *= torch.where(t >= 0, grad, 0.0).double()[:, None]
    for got, want in ((xs.grad, z @ w.double()), (ws.grad, z.t().contiguous() @ x.double())):
        least = (want.to(dtype).double() - want).norm()
        assert float((got.double() - want).norm()) <= 1.02 * float(least)
    assert float((bs.grad.double() - z.sum(0)).norm() / z.sum(0).norm()) < 2.0 ** -16


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N,V,H", [(65, 35, 64), (167, 35, 73), (300, 500, 64), (100, 5000, 128),
                                   (2000, 29, 512)])
def test_small_calls_are_off_by_their_own_rounding(dtype, N, V, H):
    """As with a split d, without being asked; two weights, one of them seldom, whose
    targets' entries would all be rounded the same way."""
    x, w, t, b, _ = make(N, V, H, dtype, seed=N)
    grad = torch.where(torch.arange(N, device="cuda") % 50 == 7, 1.0, 0.51)
    _, lse = lm.token_loss_forward(x, w, t, b)
    dx, dw, _ = lm.token_loss_backward(grad, x, w, t, lse, b)
    z = torch.softmax(x.double() @ w.double().t() + b.double(), 1)
    live = torch.nonzero(t >= 0)[:, 0]
    z[live, t[live].long()] -= 1
    z *= torch.where(t >= 0, grad, 0.0).double()[:, None]
    for got, want in ((dx, z @ w.double()), (dw, z.t().contiguous() @ x.double())):
        least = (want.to(dtype).double() - want).norm()
        assert float((got.double() - want).norm()) <= 1.02 * float(least)


def test_split_d_of_f32_changes_nothing():
    x, w, t, b, grad = make(200, 300, 64, torch.float32)
    _, lse = lm.token_loss_forward(x, w, t, b)
    got = lm.token_loss_backward(grad, x, w, t, lse, b, split_d=True)
    want = lm.token_loss_backward(grad, x, w, t, lse, b)
    assert all(torch.equal(a, c) for a, c in zip(got, want))
