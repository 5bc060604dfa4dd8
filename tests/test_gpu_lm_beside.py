"""Results written beside an input, in the same tensor."""
import pytest
import torch

from ctc_prefix_beam_amd import lm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,n", [(3, 100), (2, 3000), (900, 30)])   # each launch form
def test_attention_to_other_heads_of_the_tensor_that_q_is_from(rows, n):
    Hq, Hkv, D, page = 8, 2, 64, 16
    pages = -(-n // page)
    g = torch.Generator(device="cuda").manual_seed(n)
    c = [torch.randint(-127, 128, (pages, page, Hkv, D), generator=g, device="cuda").to(torch.int8)
         for _ in range(2)]
    s = [torch.full((pages, Hkv), 2.0 ** -6, device="cuda") for _ in range(2)]
    tables = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(rows, 1)
    lens = torch.randint(0, n + 1, (rows,), generator=g, device="cuda", dtype=torch.int32)
    qkv = torch.randn((rows, 2 * Hq + 2 * Hkv, D), generator=g, device="cuda").to(torch.bfloat16)
    for q, out in ((slice(0, Hq), slice(Hq, 2 * Hq)), (slice(0, 2 * Hq, 2), slice(1, 2 * Hq, 2))):
        both = qkv.clone()
        want, wl = lm.attention8(both[:, q].contiguous(), *c, *s, tables, lens)
        got, lse = lm.attention8(both[:, q], *c, *s, tables, lens, out=both[:, out])
        assert got.data_ptr() == both[:, out].data_ptr()
        assert torch.equal(got, want) and torch.equal(lse, wl)
        left = torch.ones(both.shape[1], dtype=torch.bool)
        left[out] = False
        assert torch.equal(both[:, left], qkv[:, left])
    with pytest.raises(ValueError, match="overlap"):
        lm.attention8(qkv[:, :Hq], *c, *s, tables, lens, out=qkv[:, 1:Hq + 1])
