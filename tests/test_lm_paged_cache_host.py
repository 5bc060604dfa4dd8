"""What a paged cache refuses when it is made, on the CPU."""
import pytest
import torch

from ctc_prefix_beam_amd import lm


@pytest.mark.parametrize("dtype", [torch.int8, torch.float8_e4m3fn])
def test_codes_of_heads_that_no_attention_reads(dtype):
    for D in (0, 8, 20, 72, 250, 272, 512, -16):
        with pytest.raises(ValueError, match="head_dim"):
            lm.PagedCache(2, 32, 1, D, dtype=dtype, device="cpu")
    for D in (16, 80, 256):
        assert lm.PagedCache(2, 32, 1, D, dtype=dtype, device="cpu").k.shape[-1] == D
    assert lm.PagedCache(2, 32, 1, 72, device="cpu").k.shape[-1] == 72   # 16 bits: a multiple of 8
