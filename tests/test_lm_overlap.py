"""Which outputs are taken to overlap an input, on the CPU: none that does is let through, and
parts of one tensor that lie beside each other are."""
import random

import pytest
import torch

from ctc_prefix_beam_amd import lm


def meets(out, t):
    try:
        lm._off(out, t, "x")
    except ValueError as e:
        assert "overlap" in str(e)
        return True
    return False


def shares(a, b):
    """Whether elements of two views of one tensor share bytes, one by one."""
    base = a.untyped_storage().data_ptr()
    got = []
    for x in (a, b):
        at = torch.zeros((), dtype=torch.int64)
        for n, s in zip(x.shape, x.stride()):
            at = at[..., None] + torch.arange(n) * s * x.itemsize
        at = (at.reshape(-1) + (x.data_ptr() - base))[:, None] + torch.arange(x.itemsize)
        got.append(set(at.reshape(-1).tolist()))
    return bool(got[0] & got[1])


def test_parts_of_a_fused_projection():
    """Heads of one tensor, as an attention takes and leaves them."""
    Hq, Hkv, D = 8, 2, 64
    qkv = torch.zeros((5, 2 * Hq + 2 * Hkv, D), dtype=torch.float16)
    q = qkv[:, :Hq]
    assert not meets(qkv[:, Hq:2 * Hq], q)
    assert not meets(q, qkv[:, Hq:2 * Hq])
    assert not meets(qkv[:, 2:2 + Hkv], qkv[:, Hq:Hq + Hkv])
    assert meets(qkv[:, Hq - 1:2 * Hq - 1], q) and meets(qkv[:, 1:Hq + 1], q)
    # heads that take turns, and halves of a head
    assert not meets(qkv[:, 1:2 * Hq:2], qkv[:, 0:2 * Hq:2])
    assert meets(qkv[:, 1:2 * Hq:2], qkv[:, 1:2 * Hq:2])
    assert not meets(qkv[:, :Hq, D // 2:], qkv[:, :Hq, :D // 2])
    assert meets(qkv[:, :Hq, D // 2 - 1:], qkv[:, :Hq, :D // 2])
    # requests that take turns, and one tensor behind the other
    assert not meets(qkv[1::2, :Hq], qkv[0:4:2, :Hq])
    assert not meets(qkv[3:, :Hq], qkv[:2, :Hq]) and meets(qkv[1:4], qkv[:3])
    # an expanded input, beside and under the output
    assert not meets(qkv[:, Hq:2 * Hq], qkv[:1, :Hq].expand(5, Hq, D))
    assert meets(qkv[:, Hq:2 * Hq], qkv[:1, Hq:Hq + 1].expand(5, Hq, D))
    assert not meets(qkv[:0], qkv) and not meets(qkv, torch.zeros_like(qkv))


@pytest.mark.parametrize("seed", range(40))
def test_views_of_any_kind(seed):
    """Random views of a few axes, steps and types: what shares a byte is never let through."""
    rng = random.Random(seed)
    found = 0
    for _ in range(200):
        base = torch.zeros(1600, dtype=torch.uint8)
        views = []
        for _ in range(2):
            dtype = rng.choice((torch.int8, torch.float16, torch.float32))
            flat = base.view(dtype)
            shape = [rng.randint(1, 4) for _ in range(rng.randint(1, 3))]
            stride = [rng.choice((0, 1, 2, 3, 4, 8, 12, 24, 36)) for _ in shape]
            top = flat.numel() - sum(s * (n - 1) for s, n in zip(stride, shape)) - 1
            views.append(flat.as_strided(shape, stride, rng.randint(0, min(top, 40))))
        real = shares(*views)
        found += real
        assert meets(*views) >= real
    assert 20 < found < 180


def test_strips_of_equal_strides_are_told_apart_exactly():
    """Views of one tensor with three axes: refused only where they share an element."""
    base = torch.zeros((4, 6, 8), dtype=torch.float16)
    rng = random.Random(1)
    for _ in range(2000):
        views = []
        for _ in range(2):
            cut = [sorted(rng.sample(range(n + 1), 2)) for n in base.shape]
            views.append(base[cut[0][0]:cut[0][1], cut[1][0]:cut[1][1], cut[2][0]:cut[2][1]])
        a, b = views
        apart = [x.storage_offset() for x in views]
        if a.shape[1:] == b.shape[1:] and min(a.shape + b.shape) > 1:
            # (strips of all requests are compared, whichever of them the two have)
            rows = [base[:, (o // 8) % 6:(o // 8) % 6 + x.shape[1], o % 8:o % 8 + x.shape[2]]
                    for o, x in zip(apart, views)]
            if not shares(*rows):
                assert not meets(a, b)
        assert meets(a, b) >= shares(a, b)
