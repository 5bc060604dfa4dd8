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
