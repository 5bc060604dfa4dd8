"""What the binding of the language-model operators does on the host, without a
GPU: the library's calls are replaced by stand-ins."""
import ctypes
import os

import pytest
import torch

from ctc_prefix_beam_amd import lm


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(lm.LIB_PATH):
        from ctc_prefix_beam_amd import build
        build.build_lm()
    return lm.lib()


class Marked:
    """A tensor's stand-in that keeps the streams it was marked as used on."""

    def __init__(self):
        self.streams = []

    def record_stream(self, stream):
        self.streams.append(stream)


def marked_cache():
    c = lm.PagedCache(2, 32, 1, 8, dtype=torch.float32, device="cpu")
    for name in ("k", "v", "tables", "pool", "lengths", "taken"):
        setattr(c, name, Marked())
    return c


@pytest.mark.parametrize("call", ["append", "release"])
def test_memory_that_a_cache_gives_up_is_kept_for_the_stream_that_reads_it(call, monkeypatch):
    """append and release leave the old lengths and `taken` to the allocator while the
    call on `stream` may not have read them yet."""
    new = lm.CachePlan(*[torch.zeros(1)] * 6)
    monkeypatch.setattr(lm, "cache_plan", lambda *a: new)
    monkeypatch.setattr(lm, "cache_release", lambda *a: (new.lengths, new.taken))
    c, stream = marked_cache(), object()
    held = [c.lengths, c.taken, c.tables, c.pool]
    if call == "append":
        c.append(None, 1, stream=stream)
    else:
        c.release(None, stream=stream)
    assert c.lengths is new.lengths and c.taken is new.taken
    assert all(t.streams == [stream] for t in held)


def test_a_cache_dropped_after_a_call_is_kept_for_the_stream_of_the_call(monkeypatch):
    monkeypatch.setattr(lm, "cache_store", lambda *a: None)
    monkeypatch.setattr(lm, "attention", lambda *a, **kw: None)
    c, stream = marked_cache(), object()
    monkeypatch.setattr(Marked, "__getitem__", lambda self, layer: None, raising=False)
    c.store(None, None, None, stream=stream)
    assert c.k.streams == [stream] and c.v.streams == [stream]
    c.attend(None, stream=stream)
    assert c.tables.streams == [stream] and c.lengths.streams == [stream]


@pytest.mark.parametrize("dtype,D", [(0, 64), (1, 72), (2, 128)])
@pytest.mark.parametrize("group", [1, 2, 3, 5, 16, 17, 40])
def test_every_part_of_a_split_row_begins_on_16_bytes(L, group, dtype, D):
    """The parts lie one after another behind the rows' prefix sums, two to a range, and
    are accessed 16 bytes at a time: an odd number of ranges shows a place that is not a
    multiple of 16 bytes."""
    n, page = 128 * 65, 16   # 65 steps of four tiles of 32 tokens (f32: 130 of 16)
    out = ctypes.c_size_t()
    assert L.ctcpb_lm_attention_workspace(lm._ATTENTION.pack(
        0, 0, 0, 0, 0, 0, 0, 0, 0, n // page, *(256, 64, 64, 64) * 2, dtype, 1, group, 1, D, 1, page,
        n // page, n, 0, 1.0), out) == 0
    tiles, ranges = -(-group // 16), 65 if dtype < 2 else 130
    places = ranges * tiles * 2
    each, rest = divmod(out.value - 256, places)   # prefix sums of one row: 256 bytes
    assert rest == 0 and each % 16 == 0
    assert each >= min(16, group) * (D + 2) * 4


def test_second_derivatives_of_the_token_loss_are_refused(monkeypatch):
    """The gradients come from the library and carry no graph of their own: a loss of them
    would lose their part without a word."""
    monkeypatch.setattr(lm, "token_loss_forward",
                        lambda x, w, t, b: ((x.detach() ** 3).sum(1), x.detach().sum(1)))
    monkeypatch.setattr(lm, "token_loss_backward",
                        lambda g, x, w, *a, **kw: (g[:, None] * 3 * x ** 2, None, None))
    x = torch.ones((2, 3), requires_grad=True)
    loss = lm.token_loss(x, torch.zeros(4, 3), torch.zeros(2, dtype=torch.int32)).sum()
    (d,) = torch.autograd.grad(loss, x, create_graph=True)
    assert torch.equal(d, torch.full_like(d, 3.0))
    with pytest.raises(RuntimeError, match="twice"):
        (loss + d.pow(2).sum()).backward()


def grad_workspace(L, rows, V, H, dtype=0, bias=256):
    out = ctypes.c_size_t()
    assert L.ctcpb_lm_loss_grad_workspace(lm._GRAD.pack(
        256, 256, bias, 256, 256, 256, 256, 256, bias, H, H, dtype, rows, V, H), out) == 0
    return out.value


@pytest.mark.parametrize("dtype,rows,V,H", [(0, 8192, 50000, 2048), (2, 2000, 9000, 1024),
                                            (2, 9000, 2000, 1024)])
def test_a_gradient_takes_little_more_than_its_d(L, dtype, rows, V, H):
    """Sums of parts of k are kept for the rows that are cut along k (808 or 848 here, in 2
    or 4 parts), not for all of the result: under a tenth of d; the partial sums of dbias,
    of 32 tokens or more each, only with a bias."""
    d = rows * (-(-V // 256) * 256) * (4 if dtype == 2 else 2)
    assert grad_workspace(L, rows, V, H, dtype, bias=0) <= d * 1.1 + 1024
    more = grad_workspace(L, rows, V, H, dtype) - grad_workspace(L, rows, V, H, dtype, bias=0)
    assert 0 < more <= -(-rows // 32) * V * 4 + 256 * 64


def test_a_split_d_has_twice_the_room_and_is_for_gradients_only(L):
    one, two = (grad_workspace(L, 1000, 5000, 512, dtype, bias=0) for dtype in (0, 256))
    d = 1000 * 5120 * 2
    assert one >= d and two >= 2 * d
    assert grad_workspace(L, 1000, 5000, 512, 258) == grad_workspace(L, 1000, 5000, 512, 2)
    out = ctypes.c_size_t()
    args = lm._LOSS.pack(256, 256, 0, 256, 256, 256, 64, 64, 256, 3, 100, 64)
    assert L.ctcpb_lm_loss_workspace(args, out) == 1
    args = lm._GRAD.pack(*[256] * 9, 64, 64, 256 + 3, 3, 100, 64)
    assert L.ctcpb_lm_loss_grad_workspace(args, out) == 1
    args = lm._GRAD.pack(*[256] * 9, 64, 64, 256, 1 << 30, 1, 64)
    assert L.ctcpb_lm_loss_grad_workspace(args, out) == 3
