"""Attention by ranges of all requests' tokens (rows longer than a workgroup takes), split
rows joined from their parts, against float64."""
import ctypes
import math

import pytest
import torch

import lm_ref_rows
from ctc_prefix_beam_amd import lm

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def make(lengths, Hq, Hkv, D, dtype, page, width, seed):
    """q, caches, tables, lengths; every slot no request owns holds NaN."""
    g = torch.Generator().manual_seed(seed)
    have = [-(-n // page) for n in lengths]
    pages = sum(have) + 1
    kc = torch.randn((pages, page, Hkv, D), generator=g).to(dtype)
    vc = torch.randn((pages, page, Hkv, D), generator=g).to(dtype)
    perm = torch.randperm(pages, generator=g).tolist()
    tables = torch.full((len(lengths), width), -1, dtype=torch.int32)
    used = torch.zeros((pages, page), dtype=torch.bool)
    at = 0
    for r, n in enumerate(lengths):
        for j in range(have[r]):
            tables[r, j] = perm[at]
            used[perm[at], :min(page, n - j * page)] = True
            at += 1
    kc[~used], vc[~used] = math.nan, math.nan
    q = (2 * torch.randn((len(lengths), Hq, D), generator=g)).to(dtype)
    lens = torch.tensor(lengths, dtype=torch.int32)
    return tuple(t.cuda() for t in (q, kc, vc, tables, lens))


def by_ranges(q, kc, tables, window):
    """Whether a call takes this path: it alone has a workspace."""
    out = ctypes.c_size_t()
    R, Hq, D = q.shape
    _, page, Hkv, _ = kc.shape
    width = tables.shape[1]
    lm._check(lm.lib().ctcpb_lm_attention_workspace(lm._ATTENTION.pack(
        0, 0, 0, 0, 0, 0, 0, 0, 0, width, *(0, 0, 0, 0) * 2, lm._TYPES[q.dtype], R, Hq, Hkv, D,
        kc.shape[0], page, width, 0, window, 1.0), out))
    return out.value > 0


def check(q, kc, vc, tables, lens, window=0):
    assert by_ranges(q, kc, tables, window)
    page, D = kc.shape[1], q.shape[2]
    out, lse = lm.attention(q, kc, vc, tables, lens, window=window)
    want = lm_ref_rows.attention(q, kc, vc, tables, lens, D ** -0.5, window, page)
    to, tl = lm_ref_rows.tolerances(*want, D, q.dtype)
    out, lse = out.cpu().double(), lse.cpu().double()
    dead = want[1] == -math.inf
    assert torch.isfinite(out).all() and torch.equal(lse == -math.inf, dead)
    assert ((out - want[0]).abs() <= to).all(), float(((out - want[0]).abs() - to).max())
    assert ((lse - want[1]).abs()[~dead] <= tl[~dead]).all()


LONG = [9000, 0, 1, 33, 5003, 128, 31, 2500]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Hq,Hkv,D", [(1, 1, 64), (3, 3, 64), (3, 1, 72), (5, 1, 128), (10, 2, 64),
                                      (17, 1, 64), (40, 1, 128), (20, 1, 136), (34, 2, 64),
                                      (9, 3, 256)])
def test_rows_split_between_workgroups(dtype, Hq, Hkv, D):
    """Odd head groups, several head tiles and a last one with few heads; a group of
    threads to each row and head, or several that share its parts."""
    check(*make(LONG, Hq, Hkv, D, dtype, 16, 600, Hq + D))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Hq,Hkv", [(17, 1), (5, 5), (33, 1)])
def test_many_heads_joined_by_one_group_of_threads_each(dtype, Hq, Hkv):
    rows = 1025 // Hq + 5
    lengths = [(379 * r) % 3001 for r in range(rows)]
    check(*make(lengths, Hq, Hkv, 64, dtype, 32, 100, Hq))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("window", [2500, 4001])
@pytest.mark.parametrize("Hq,Hkv", [(3, 3), (20, 1)])
def test_windows_that_begin_inside_a_tile(dtype, window, Hq, Hkv):
    check(*make([9000, 0, 2499, 2501, 7777, 4003], Hq, Hkv, 64, dtype, 16, 600, window), window)


@pytest.mark.parametrize("lengths,Hq,Hkv", [([300, 77, 500], 4, 2), ([9000, 700], 3, 1),
                                            ([40000], 8, 2)])
@pytest.mark.parametrize("window", [0, 450])
def test_f32_outputs_in_the_2_norm(lengths, Hq, Hkv, window):
    """Products of 64 terms reach 32 before their scale of 1 / 8: a rounding is 0.29 of 2^-19 at
    the root mean square, some 32 of them in a chain that large, so a score, and with it the
    logarithm of a probability, is off by 0.29 2^-19 sqrt(32) / 8 = 0.2 2^-19; sums in chains
    of tiles, the exponentials and the division by 2^-22 at most.  Twice that is allowed."""
    q, kc, vc, tables, lens = make(lengths, Hq, Hkv, 64, torch.float32, 16, 2600, len(lengths))
    out, lse = lm.attention(q, kc, vc, tables, lens, window=window)
    want = lm_ref_rows.attention(q, kc, vc, tables, lens, 0.125, window, 16)
    tol = 2 * (0.2 * 2.0 ** -19 + 2.0 ** -22)
    assert float((out.cpu().double() - want[0]).norm() / want[0].norm()) <= tol
    assert ((lse.cpu().double() - want[1]).abs() <= 4 * tol + 2.0 ** -23 * want[1].abs()).all()
