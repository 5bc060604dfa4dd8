"""Host-side checks of the 8-bit operators that need no GPU: every refused argument is refused
with its status before the device is touched, and sizes of workspaces."""
import ctypes
import os

import pytest
import torch

from ctc_prefix_beam_amd import lm

P, N = 256, 0   # addresses that are never dereferenced


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(lm.LIB_PATH):
        from ctc_prefix_beam_amd import build
        build.build_lm()
    return lm.lib()


def cache(data=P, page=2048, token=128, head=64):
    return data, page, token, head


def scales(data=P, page=2, head=1):
    return data, page, head


def cache8(call, k=P, v=P, slots=P, st=128, sh=64, kc=cache(), vc=cache(), ks=scales(), vs=scales(),
           dtype=0, code=0, T=3, pages=4, page=16, H=2, D=64):
    return call(lm._CACHE8.pack(k, v, slots, st, sh, st, sh, *kc, *vc, *ks, *vs, dtype, code, T,
                                pages, page, H, D), None)


@pytest.mark.parametrize("kw", [
    dict(dtype=3), dict(dtype=-1), dict(code=2), dict(code=-1), dict(k=N), dict(v=N), dict(slots=N),
    dict(T=-1), dict(vc=cache(0)), dict(kc=cache(0)), dict(pages=0), dict(page=3), dict(H=0),
    dict(D=0), dict(st=-1), dict(sh=-1), dict(pages=1 << 28), dict(kc=cache(token=-1)),
    dict(H=1 << 13, D=1 << 12), dict(ks=scales(0)), dict(vs=scales(0)), dict(ks=scales(page=-1)),
    dict(vs=scales(head=-1))])
def test_store_and_load_refusals(L, kw):
    for call in (L.ctcpb_lm_cache_store8, L.ctcpb_lm_cache_load8):
        assert cache8(call, **kw) == 1
        assert L.ctcpb_lm_last_error().decode() != ""


def test_more_tokens_than_a_launch_has_threads_for(L):
    wide = dict(k=1 << 20, v=1 << 20, D=128, st=8192, sh=128)
    for kw in (dict(page=16), dict(page=32), dict(page=256), dict(page=16, D=64)):
        assert cache8(L.ctcpb_lm_cache_store8, T=(1 << 27), H=64, **{**wide, **kw}) == 3
        assert "too many tokens" in L.ctcpb_lm_last_error().decode()


def test_no_tokens(L):
    for call in (L.ctcpb_lm_cache_store8, L.ctcpb_lm_cache_load8):
        assert cache8(call, T=0, k=N, v=N, slots=N) == 0


def attend(L, dtype=0, code=0, q=P, sr=128, sh=64, kc=cache(), vc=cache(), ks=scales(), vs=scales(),
           pages=4, page=16, tables=P, stride=8, width=8, lengths=P, rows=3, Hq=4, Hkv=2, D=64,
           max_len=0, window=0, out=P, ws=P, ws_bytes=1 << 40):
    return L.ctcpb_lm_attention8(lm._ATTENTION8.pack(
        q, tables, lengths, out, N, sr, sh, sr, sh, stride, *kc, *vc, dtype, rows, Hq, Hkv, D,
        pages, page, width, max_len, window, 1.0, *ks, *vs, code), ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=7), 1), (dict(code=2), 1), (dict(rows=-1), 1), (dict(Hq=3), 1), (dict(Hkv=0), 1),
    (dict(D=0), 1), (dict(D=72), 1), (dict(D=272), 3), (dict(max_len=-1), 1), (dict(window=-1), 1),
    (dict(page=6), 1), (dict(pages=0), 1), (dict(stride=2), 1), (dict(sr=-1), 1), (dict(q=N), 1),
    (dict(out=N), 1), (dict(lengths=N), 1), (dict(tables=N), 1), (dict(kc=cache(0)), 1),
    (dict(vc=cache(0)), 1), (dict(kc=cache(264)), 1), (dict(vc=cache(token=72)), 1),
    (dict(ks=scales(0)), 1), (dict(vs=scales(0)), 1), (dict(vs=scales(page=-2)), 1),
    (dict(width=4096, stride=4096, ws=N), 1), (dict(width=4096, stride=4096, ws_bytes=16), 2),
    (dict(rows=1 << 30, Hq=64, Hkv=64), 3), (dict(rows=1 << 24), 3), (dict(kc=cache(page=1 << 32)), 3),
    (dict(vc=cache(token=(1 << 23) + 16)), 3), (dict(ks=scales(page=1 << 30)), 3),
    (dict(vs=scales(page=1 << 62)), 3)])
def test_attention_refusals(L, kw, code):
    assert attend(L, **kw) == code
    assert L.ctcpb_lm_last_error().decode() != ""


@pytest.mark.parametrize("group", [1, 3, 16, 17, 40])
@pytest.mark.parametrize("D", [48, 128, 256])
def test_attention_workspace(L, group, D):
    """None for rows that are not split, and parts that begin on 16 bytes."""
    def ws(rows, n, window=0):
        out = ctypes.c_size_t(7)
        assert L.ctcpb_lm_attention8_workspace(lm._ATTENTION8.pack(
            N, N, N, N, N, 0, 0, 0, 0, -(-n // 16), *cache(), *cache(), 0, rows, group, 1, D, 1, 16,
            -(-n // 16), n, window, 1.0, N, 0, 0, N, 0, 0, 0), out) == 0
        return out.value
    assert ws(0, 0) == 0 and ws(5, 300) == 0
    one = ws(1, 131072)
    assert one > 256 and (one - 256) % 32 == 0
    assert ws(1, 131072, window=64) == 0
    assert attend(L, rows=0, q=N, out=N, lengths=N, tables=N) == 0


def test_quantize_refusals(L):
    def quantize(x=P, codes=P, s=P, sx=64, sc=64, dtype=0, rows=3, H=64):
        return L.ctcpb_lm_quantize_rows(lm._QUANTIZE.pack(x, codes, s, sx, sc, dtype, rows, H), None)
    for kw in (dict(x=N), dict(codes=N), dict(s=N), dict(sx=-1), dict(sc=63), dict(dtype=3),
               dict(rows=-1), dict(H=0), dict(H=(1 << 30) + 1, sc=1 << 31)):
        assert quantize(**kw) == 1, kw
    assert quantize(rows=0, x=N, codes=N, s=N) == 0


def linear(L, x=P, xs=N, w=P, wscale=P, out=P, sx=64, sw=64, so=100, xt=0, dtype=0, rows=90, M=100,
           H=64, flags=0, ws=P, ws_bytes=1 << 40):
    return L.ctcpb_lm_linear8(lm._LINEAR8.pack(x, xs, w, wscale, N, out, sx, sw, so, xt, dtype, rows,
                                               M, H, flags), ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=N), 1), (dict(w=N), 1), (dict(wscale=N), 1), (dict(out=N), 1), (dict(xt=3), 1),
    (dict(xt=4), 1), (dict(xt=1), 1), (dict(xt=-1), 1), (dict(dtype=3), 1), (dict(rows=-1), 1), (dict(M=0), 1),
    (dict(H=0), 1), (dict(sx=-1), 1), (dict(sw=-1), 1), (dict(so=99), 1), (dict(flags=2), 1),
    (dict(H=131072), 3), (dict(rows=1 << 30, M=1 << 30, so=1 << 30), 3), (dict(ws=N), 1),
    (dict(ws=264), 1), (dict(ws_bytes=8), 2)])
def test_linear_refusals(L, kw, code):
    assert linear(L, **kw) == code
    assert L.ctcpb_lm_last_error().decode() != ""


def test_linear_workspace(L):
    def size(x=P, w=P, sx=64, sw=64, xt=0, rows=1000, M=5000, H=64, flags=0):
        out = ctypes.c_size_t(3)
        assert L.ctcpb_lm_linear8_workspace(lm._LINEAR8.pack(
            x, N, w, N, N, N, sx, sw, M, xt, 0, rows, M, H, flags), out) == 0
        return out.value
    assert size(rows=16, H=512, sx=512, sw=512) == 0   # few rows: one launch
    codes, one = -(-1000 * 64 // 256) * 256, -(-4000 // 256) * 256
    assert size() == codes + one                       # x as codes, and their scales
    assert size(xt=3) == 0                             # everything in place
    assert size(xt=3, x=P + 8) == size(xt=3, sx=72) == codes
    assert size(xt=3, w=P + 8) == size(xt=3, sw=72) == 5000 * 64
    # rows that end inside 16 bytes: x's codes need zeros there, w's to be there
    assert size(xt=3, H=60) == codes + 5000 * 64 and size(xt=3, H=60, flags=1) == codes
    assert size(rows=0) == 0
    # few rows and long sums: parts of them, as whole numbers
    assert size(xt=3, rows=64, M=100, H=8192, sx=8192, sw=8192) % (64 * 100 * 4) == 0
    assert linear(L, rows=0, x=N, w=N, wscale=N, out=N, ws=N) == 0


def test_readable_rows():
    """The last row counts: where it ends with its memory, it cannot be read past its end."""
    t = torch.zeros((4, 48), dtype=torch.int8)
    assert lm._readable(t[:, :40], 48, 4, 40)
    assert lm._readable(t, 48, 4, 48)
    assert not lm._readable(t[:, 8:], 48, 4, 40)
    assert lm._readable(t[:3, 8:], 48, 3, 40)
    assert not lm._readable(torch.zeros((4, 40), dtype=torch.int8), 40, 4, 40)


def test_a_cache_of_codes():
    c = lm.PagedCache(2, 32, 3, 64, dtype=torch.int8, page_size=8, layers=2, device="cpu")
    assert c.k.shape == c.v.shape == (2, 8, 8, 3, 64) and c.k.dtype == torch.int8
    assert c.k[0].stride() == (3 * 8 * 64, 64, 8 * 64, 1)       # a page's head lies together
    assert c.k_scale.shape == c.v_scale.shape == (2, 8, 3)
    assert (c.k_scale == 0).all() and (c.v_scale == 0).all()
    assert lm.PagedCache(2, 32, 3, 64, device="cpu").k_scale is None
    with pytest.raises(ValueError, match="int8"):
        lm.PagedCache(2, 32, 3, 64, device="cpu").load(None)
