"""Host-side checks of libctcpb_lm.so that need no GPU: the symbols of
include/ctcpb_lm.h are exported, and every refused argument is refused with its
status before the device is touched."""
import ctypes
import os
import re

import pytest

from ctc_prefix_beam_amd import lm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ctcpb_lm.h")
P, N = 256, 0   # addresses that are never dereferenced


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(lm.LIB_PATH):
        from ctc_prefix_beam_amd import build
        build.build_lm()
    return lm.lib()


def test_every_declared_symbol_is_exported(L):
    text = open(HEADER).read()
    names = re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(ctcpb_lm_\w+)\s*\(", text, re.M)
    assert set(names) == set(lm.EXPORTS), names
    for n in names:
        assert hasattr(L, n), n


def plan(L, lengths=P, counts=P, rows=4, tables=P, stride=8, width=8, pool=P, pool_size=9, taken=P,
         page=16, slots=P, positions=P, cap=5, starts=P, out=P, now=P, status=P):
    return L.ctcpb_lm_cache_plan(lm._PLAN.pack(
        lengths, counts, tables, pool, taken, slots, positions, starts, out, now, status, stride,
        rows, width, pool_size, page, cap), None)


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(page=0), dict(page=2), dict(page=24), dict(page=512), dict(stride=7),
    dict(width=-1), dict(width=1 << 27, stride=1 << 27), dict(pool_size=-1), dict(cap=-1),
    dict(cap=(1 << 30) + 1), dict(lengths=N), dict(counts=N), dict(tables=N), dict(pool=N),
    dict(taken=N), dict(slots=N), dict(positions=N), dict(starts=N), dict(out=N), dict(now=N),
    dict(status=N)])
def test_plan_refusals(L, kw):
    assert plan(L, **kw) == 1
    assert L.ctcpb_lm_last_error().decode() != ""


def test_release_refusals(L):
    def release(fin=P, lengths=P, rows=4, tables=P, stride=8, width=8, pool=P, pool_size=9, taken=P,
                page=16, out=P, now=P):
        return L.ctcpb_lm_cache_release(lm._RELEASE.pack(
            fin, lengths, tables, pool, taken, out, now, stride, rows, width, pool_size, page), None)
    for kw in (dict(fin=N), dict(lengths=N), dict(tables=N), dict(pool=N), dict(taken=N),
               dict(out=N), dict(now=N), dict(page=5), dict(rows=-1), dict(pool_size=-2)):
        assert release(**kw) == 1


def cache(data=256, page=2048, token=128, head=64):
    return data, page, token, head


def test_store_refusals(L):
    def store(dtype=0, k=P, st=128, sh=64, v=P, slots=P, T=3, kc=cache(), vc=cache(), pages=4,
              page=16, H=2, D=64):
        return L.ctcpb_lm_cache_store(lm._STORE.pack(
            k, v, slots, st, sh, st, sh, *kc, *vc, dtype, T, pages, page, H, D), None)
    for kw in (dict(dtype=3), dict(dtype=-1), dict(k=N), dict(v=N), dict(slots=N), dict(T=-1),
               dict(vc=cache(0)), dict(kc=cache(0)), dict(pages=0), dict(page=3),
               dict(H=0), dict(D=0), dict(st=-1), dict(pages=1 << 28), dict(kc=cache(token=-1)),
               dict(H=1 << 20, D=1 << 20)):
        assert store(**kw) == 1, kw
    assert store(T=0, k=N, v=N, slots=N) == 0


def attend(L, dtype=0, q=P, sr=128, sh=64, kc=cache(), vc=cache(), pages=4, page=16, tables=P,
           stride=8, width=8, lengths=P, rows=3, Hq=4, Hkv=2, D=64, max_len=0, window=0, out=P,
           ws=P, ws_bytes=1 << 40):
    return L.ctcpb_lm_attention(lm._ATTENTION.pack(
        q, tables, lengths, out, N, sr, sh, sr, sh, stride, *kc, *vc, dtype, rows, Hq, Hkv, D,
        pages, page, width, max_len, window, 1.0), ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=7), 1), (dict(rows=-1), 1), (dict(Hq=3), 1), (dict(Hkv=0), 1), (dict(Hq=0), 1),
    (dict(D=0), 1), (dict(D=60), 1), (dict(D=264), 3), (dict(max_len=-1), 1), (dict(window=-1), 1),
    (dict(page=6), 1), (dict(pages=0), 1), (dict(stride=2), 1), (dict(sr=-1), 1), (dict(q=N), 1),
    (dict(out=N), 1), (dict(lengths=N), 1), (dict(tables=N), 1), (dict(kc=cache(0)), 1),
    (dict(vc=cache(0)), 1), (dict(kc=cache(264)), 1), (dict(vc=cache(token=63)), 1),
    (dict(width=4096, stride=4096, ws=N), 1), (dict(width=4096, stride=4096, ws_bytes=16), 2),
    (dict(rows=1 << 30, Hq=64, Hkv=64), 3)])
def test_attention_refusals(L, kw, code):
    assert attend(L, **kw) == code
    assert L.ctcpb_lm_last_error().decode() != ""


def test_attention_workspace(L):
    def ws(rows, Hq, Hkv, D, n, window=0, dtype=0):
        out = ctypes.c_size_t(7)
        rc = L.ctcpb_lm_attention_workspace(lm._ATTENTION.pack(
            N, N, N, N, N, 0, 0, 0, 0, -(-n // 16), *cache(), *cache(), dtype, rows, Hq, Hkv, D, 1,
            16, -(-n // 16), n, window, 1.0), out)
        return rc, out.value
    assert ws(0, 4, 2, 64, 0) == (0, 0)
    rc, one = ws(1, 32, 8, 128, 131072)
    assert rc == 0 and one > 0
    assert ws(1, 32, 8, 128, 131072, window=64)[1] < one   # a window bounds the length
    assert ws(1, 3, 2, 64, 100)[0] == 1
    assert attend(L, rows=0, q=N, out=N, lengths=N, tables=N) == 0


def loss(L, dtype=0, x=P, sx=64, w=P, sw=64, targets=P, rows=3, V=100, H=64, out=P, lse=P, ws=P,
         ws_bytes=1 << 40):
    return L.ctcpb_lm_loss(lm._LOSS.pack(x, w, N, targets, out, lse, sx, sw, dtype, rows, V, H), ws,
                           ws_bytes, None)


def grad(L, dtype=0, g=P, x=P, sx=64, w=P, sw=64, targets=P, lse=P, rows=3, V=100, H=64, dx=P, dw=P,
         ws=P, ws_bytes=1 << 40):
    return L.ctcpb_lm_loss_grad(lm._GRAD.pack(x, w, N, targets, g, lse, dx, dw, N, sx, sw, dtype,
                                              rows, V, H), ws, ws_bytes, None)


SIZES = [(dict(dtype=9), 1), (dict(rows=-1), 1), (dict(V=0), 1), (dict(H=0), 1), (dict(sx=63), 1),
         (dict(sw=63), 1), (dict(H=(1 << 20) + 8, sx=1 << 21, sw=1 << 21), 3),
         (dict(rows=1 << 30, V=1 << 30), 3), (dict(x=N), 1), (dict(w=N), 1), (dict(targets=N), 1),
         (dict(lse=N), 1), (dict(ws=N), 1), (dict(ws=264), 1),
         (dict(ws_bytes=8), 2)]


@pytest.mark.parametrize("kw,code", SIZES + [(dict(out=N), 1)])
def test_loss_refusals(L, kw, code):
    assert loss(L, **kw) == code
    assert L.ctcpb_lm_last_error().decode() != ""


@pytest.mark.parametrize("kw,code", SIZES + [(dict(g=N), 1), (dict(dx=8), 1),
                                             (dict(dw=8), 1)])
def test_loss_grad_refusals(L, kw, code):
    assert grad(L, **kw) == code
    assert L.ctcpb_lm_last_error().decode() != ""


def test_missing_arguments(L):
    out = ctypes.c_size_t()
    for name in lm.EXPORTS[:-1]:
        f = getattr(L, name)
        rest = {2: (None,), 4: (P, 1 << 30, None)}[len(f.argtypes)]
        if name.endswith("workspace"):
            rest = (out,)
            assert f(lm._LOSS.pack(*[P] * 6, 64, 64, 0, 1, 2, 64) + bytes(300), None) == 1
        assert f(None, *rest) == 1, name
    assert "args" in L.ctcpb_lm_last_error().decode()


def test_loss_workspaces(L):
    def size(what, x=256, sx=64, H=64, rows=1000, V=5000, dtype=0):
        out = ctypes.c_size_t(3)
        pack = lm._LOSS if what == "loss" else lm._GRAD
        ptrs = [N] * (4 if what == "loss" else 7)
        f = getattr(L, f"ctcpb_lm_{what}_workspace")
        assert f(pack.pack(x, 256, *ptrs, sx, max(H, 64), dtype, rows, V, H), out) == 0
        return out.value
    for what in ("loss", "loss_grad"):
        one = size(what)
        assert one > 0 and one % 256 == 0
        # rows that are not 16-byte aligned are copied: x of 1000 x 64 16-bit values
        assert size(what, x=258) == size(what, sx=65) == one + 128000
    # the gradient's workspace holds a piece of the vocabulary, not all of it
    many = size("loss_grad", rows=100000, V=50000)
    assert many < 100000 * 50000 * 2 / 4
    assert loss(L, rows=0, x=N, w=N, targets=N, out=N, lse=N, ws=N) == 0
    assert grad(L, dx=N, dw=N, x=N, w=N) == 0
