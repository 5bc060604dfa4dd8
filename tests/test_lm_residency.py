"""The launches count on as many workgroups sharing a CU as its LDS and the kernels' registers
allow: the built kernels' own notes have to agree."""
import os
import re

import pytest

from code_object import kernels
from ctc_prefix_beam_amd import lm

LDS, VGPRS = 160 * 1024, 512


@pytest.fixture(scope="module")
def built():
    if not os.path.exists(lm.LIB_PATH):
        from ctc_prefix_beam_amd import build
        build.build_lm()
    return kernels(lm.LIB_PATH)


def test_product_kernels_share_a_cu_as_the_cuts_count_on(built):
    """Tiles of 64 x 64 go four to a CU, of 128 x 128 two, of 256 x 256 one."""
    seen = set()
    for name, k in built.items():
        m = re.search(r"gemm_kernelI(\w+?)Li(\d+)ELi(\d+)ELi(\d+)ELi(\d+)E", name)
        if not m:
            continue
        bm, waves = int(m[2]), int(m[4]) * int(m[5])
        want = {64: 4, 128: 2, 256: 1}[bm]
        seen.add((m[1], bm))
        assert want * k[".group_segment_fixed_size"] <= LDS, name
        regs = -(-k[".vgpr_count"] // 8) * 8   # (with those for sums)
        assert VGPRS // regs * 4 // waves >= want, name
    assert {("a", 64), ("a", 128), ("a", 256)} <= seen and len(seen) >= 10
