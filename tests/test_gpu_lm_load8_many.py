"""Reading back more values than a launch has threads for."""
import pytest
import torch

from ctc_prefix_beam_amd import lm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,T", [(100, 700000), (104, 5300000)])   # single values, and pieces of 16 bytes
def test_more_values_than_threads(D, T):
    H, page, pages = 4, 16, 40
    g = torch.Generator(device="cuda").manual_seed(D)
    codes = torch.randint(-127, 128, (2, pages, page, H, D), generator=g, device="cuda").to(torch.int8)
    scales = torch.exp2(torch.randint(-9, 3, (2, pages, H), generator=g, device="cuda").float())
    slots = torch.randint(-1, pages * page, (T,), generator=g, device="cuda", dtype=torch.int32)
    assert T * H * (D if D % 8 else D // 8) > 1 << 28
    k, v = lm.cache_load8(slots, *codes, *scales)
    # (a value is a code times a power of two: exact in bfloat16)
    every = (codes.float() * scales[:, :, None, :, None]).to(torch.bfloat16).flatten(1, 2)
    none = slots < 0
    for a in range(0, T, 1 << 17):
        at = slots[a:a + (1 << 17)].long()
        for got, x in zip((k, v), every):
            want = torch.where(none[a:a + (1 << 17), None, None], 0.0, x[at.clamp(min=0)])
            assert torch.equal(got[a:a + (1 << 17)], want.to(torch.bfloat16)), a
