"""The 8-bit operators carry no gradients: whatever tensor asks for one is refused, a scale or a
result to write to as well as an input, but under torch.no_grad()."""
import pytest
import torch

from ctc_prefix_beam_amd import lm

pytestmark = pytest.mark.gpu


def tensors():
    zeros = lambda *shape, dtype=torch.float32: torch.zeros(shape, dtype=dtype, device="cuda")   # noqa: E731
    cache = dict(k_cache=zeros(2, 16, 1, 64, dtype=torch.float8_e4m3fn),
                 v_cache=zeros(2, 16, 1, 64, dtype=torch.float8_e4m3fn), k_scale=zeros(2, 1),
                 v_scale=zeros(2, 1))
    slots = dict(slots=zeros(3, dtype=torch.int32))
    return dict(
        cache_store8=dict(k=zeros(3, 1, 64), v=zeros(3, 1, 64), slots=slots["slots"] - 1, **cache),
        cache_load8=dict(**slots, **cache),
        attention8=dict(q=zeros(3, 2, 64), **cache, tables=zeros(3, 1, dtype=torch.int32),
                        lengths=zeros(3, dtype=torch.int32), out=zeros(3, 2, 64)),
        quantize_rows=dict(x=zeros(3, 32)),
        linear8=dict(x=zeros(3, 32), w=zeros(5, 32, dtype=torch.int8), w_scale=zeros(5),
                     bias=zeros(5), out=zeros(3, 5)))


CASES = [(f, n) for f, names in dict(
    cache_store8=("k", "v", "k_cache", "v_cache", "k_scale", "v_scale"),
    cache_load8=("k_cache", "v_cache", "k_scale", "v_scale"),
    attention8=("q", "k_cache", "v_cache", "k_scale", "v_scale", "out"), quantize_rows=("x",),
    linear8=("x", "w_scale", "bias", "out")).items() for n in names]


@pytest.mark.parametrize("f,name", CASES)
def test_refused(f, name):
    kw = tensors()[f]
    getattr(lm, f)(**kw)
    kw[name] = kw[name].clone().requires_grad_()
    with pytest.raises(ValueError, match=f"{f} carries no gradients"):
        getattr(lm, f)(**kw)
    with torch.no_grad():
        getattr(lm, f)(**kw)


def test_scales_of_codes_as_input():
    kw = tensors()["linear8"]
    kw["x"], kw["x_scale"], kw["out"] = kw["x"].to(torch.int8), kw["x"][:, 0].clone(), None
    lm.linear8(**kw)
    kw["x_scale"].requires_grad_()
    with pytest.raises(ValueError, match="gradients"):
        lm.linear8(**kw)
