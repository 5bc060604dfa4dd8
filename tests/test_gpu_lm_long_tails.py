"""Attention where one token takes most of the weight and the rest of the output comes from
a long tail of small probabilities."""
import pytest
import torch

import lm_ref_rows
from ctc_prefix_beam_amd import lm

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def make(rows, n, heads, D, dtype, depth, spread, seed, page=16):
    """Rows that share their pages.  Token 0 scores 0 with a value of 0, the others -depth
    and up to `spread` less with values in [0.5, 1]: scores are exact, all terms of the
    output positive."""
    g = torch.Generator().manual_seed(seed)
    pages = -(-n // page)
    k = torch.zeros((pages * page, heads, D))
    v = 0.5 + 0.5 * torch.rand((pages * page, heads, D), generator=g)
    k[:, :, 3] = -depth - spread * torch.rand((pages * page, heads), generator=g)
    k[0], v[0] = 0.0, 0.0
    k, v = k.to(dtype), v.to(dtype)
    q = torch.zeros((rows, heads, D), dtype=dtype)
    q[:, :, 3] = 1.0
    perm = torch.randperm(pages, generator=g)
    kc, vc = torch.empty((2, pages, page, heads, D), dtype=dtype)
    kc[perm], vc[perm] = k.view(pages, page, heads, D), v.view(pages, page, heads, D)
    s, vv = k[:n, :, 3].double(), v[:n].double()
    p = torch.exp(s)
    want = torch.stack([(p[:, h, None] * vv[:, h]).sum(0) / p[:, h].sum() for h in range(heads)])
    lse = torch.log(p.sum(0))
    tables = perm.to(torch.int32)[None].expand(rows, pages).contiguous()
    lens = torch.full((rows,), n, dtype=torch.int32)
    return [t.cuda() for t in (q, kc, vc, tables, lens)], want, lse


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,n,heads,D", [
    (1, 300, 2, 64), (3, 2000, 1, 128), (2, 900, 1, 256),      # a workgroup to a row and head
    (520, 500, 8, 64),                                         # a wave to each
    (1, 5000, 2, 64), (1, 65536, 1, 64), (2, 131071, 1, 128)])  # ranges
@pytest.mark.parametrize("depth,spread", [(17.0, 0.0), (17.5, 0.0), (9.0, 9.0), (5.0, 18.0)])
def test_tail_of_small_probabilities(dtype, rows, n, heads, D, depth, spread):
    """Every term is positive, so errors relative to the probabilities are relative to the
    output: 2^-17 for the exponentials and 2^-17 for two-part probabilities, 2^-24 for
    each of the n / 32 additions of a tile and of 64 joins; a probability's smallest part
    may be off by 2^-40 of the largest probability (16-bit types), and the output by its
    rounding."""
    a, want, lse = make(rows, n, heads, D, dtype, depth, spread, n + rows)
    out, got = lm.attention(*a, scale=1.0)
    out, got = out.cpu().double(), got.cpu().double()
    rel = 2.0 ** -16 + (n / 32 + 64) * 2.0 ** -24
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
    tol = want.abs() * (rel + lm_ref_rows.ULP[dtype]) + n * 2.0 ** -40 + tiny
    off = (out - want).abs() - tol
    assert (off <= 0).all(), float(((out - want).abs() / want.abs().clamp(min=1e-9)).max())
    assert ((got - lse).abs() <= rel + 2.0 ** -22).all()
