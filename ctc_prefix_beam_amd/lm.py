"""Operators for rescoring N-best lists with a language model on MI355X.

Thin Python binding of ``libctcpb_lm.so`` (C ABI in ``include/ctcpb_lm.h``):
the pages and slots of a paged key/value cache from device-resident lengths
(``cache_plan``, ``cache_release``), the store of new tokens' keys and values
(``cache_store``), the attention of one new token per request over the cache
(``attention``), and token losses over a large vocabulary without keeping the
logits, with their gradients (``token_loss``).  ``PagedCache`` holds the tensors
of a cache.  The same in 8 bits: a cache of int8 or float8_e4m3fn codes with a scale
for each page and head (``cache_store8``, ``cache_load8``, ``attention8``), and linear
layers of int8 weights with a scale for each channel (``quantize_rows``, ``linear8``);
these carry no gradients.  Every step runs in the library's HIP kernels; PyTorch provides
device memory and the current stream.  A call's `stream` (a torch stream, default
the current one) is where it runs: its inputs have to be ready there, and its
results are.  If the library is missing the calls raise; there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
from typing import NamedTuple

import torch

from . import _check_dev

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libctcpb_lm.so")

EXPORTS = ("ctcpb_lm_cache_plan", "ctcpb_lm_cache_release", "ctcpb_lm_cache_store",
           "ctcpb_lm_attention_workspace", "ctcpb_lm_attention", "ctcpb_lm_loss_workspace",
           "ctcpb_lm_loss", "ctcpb_lm_loss_grad_workspace", "ctcpb_lm_loss_grad",
           "ctcpb_lm_cache_store8", "ctcpb_lm_cache_load8", "ctcpb_lm_attention8_workspace",
           "ctcpb_lm_attention8", "ctcpb_lm_quantize_rows", "ctcpb_lm_linear8_workspace",
           "ctcpb_lm_linear8", "ctcpb_lm_last_error")
NO_PAGE, NO_ENTRY, NO_SLOT = 1, 2, 4   # status bits of cache_plan
_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_CODES = {torch.int8: 0, torch.float8_e4m3fn: 1}
_CODES_X = 3     # CTCPB_LM_CODES
_READABLE = 1    # CTCPB_LM_READABLE
_SPLIT_D = 256   # CTCPB_LM_SPLIT_D

# The argument structures of include/ctcpb_lm.h, in order (native sizes and
# alignment): a call packs them once instead of converting each argument.
_PLAN = struct.Struct("11Pq5i4x")
_RELEASE = struct.Struct("7Pq4i")
_STORE = struct.Struct("3P4qP3qP3q6i")
_ATTENTION = struct.Struct("5P5qP3qP3q10if4x")
_LOSS = struct.Struct("6P2q4i")
_GRAD = struct.Struct("9P2q4i")
_CACHE8 = struct.Struct("3P4qP3qP3qP2qP2q7i4x")
_ATTENTION8 = struct.Struct(_ATTENTION.format + "P2qP2qi4x")
_QUANTIZE = struct.Struct("3P2q3i4x")
_LINEAR8 = struct.Struct("6P3q6i")

_lib = None


def lib():
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with ctc_prefix_beam_amd.build")
        L = ctypes.CDLL(LIB_PATH)
        p, sz = ctypes.c_void_p, ctypes.c_size_t
        args = ctypes.c_char_p   # the packed structure
        for name in ("cache_plan", "cache_release", "cache_store", "cache_store8", "cache_load8",
                     "quantize_rows"):
            getattr(L, "ctcpb_lm_" + name).argtypes = [args, p]
        for name in ("attention", "loss", "loss_grad", "attention8", "linear8"):
            getattr(L, f"ctcpb_lm_{name}_workspace").argtypes = [args, ctypes.POINTER(sz)]
            getattr(L, "ctcpb_lm_" + name).argtypes = [args, p, sz, p]
        for name in EXPORTS[:-1]:   # all but the string getter
            getattr(L, name).restype = ctypes.c_int
        L.ctcpb_lm_last_error.restype = ctypes.c_char_p
        L.ctcpb_lm_last_error.argtypes = []
        _lib = L
    return _lib


def _check(rc: int):
    if rc != 0:
        msg = lib().ctcpb_lm_last_error().decode()
        if rc == 1:
            raise ValueError(msg)
        raise RuntimeError(f"ctcpb_lm error {rc}: {msg}")


def _pack(layout, *values):
    """The argument structure of a call; numbers that it cannot hold are refused."""
    try:
        return layout.pack(*values)
    except struct.error as e:
        raise ValueError(f"an argument is not a number in its range: {e}") from None


_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


class _Other:
    """Memory for a call on another stream than the current one: made on the
    current stream, which the other one waits for (the memory may have been in
    use there until now), and marked as used by the other one, so that it is not
    handed out again while the call still runs."""

    def __init__(self, stream, index):
        self.stream, self.current = stream, torch.cuda.current_stream(index)

    def __call__(self, shape, dtype, device):
        t = torch.empty(shape, dtype=dtype, device=device)
        self.stream.wait_stream(self.current)
        t.record_stream(self.stream)
        return t


def _on(stream, index):
    """(hipStream_t, allocator) of a call on `stream` (None: the current one)
    with tensors on GPU `index`, which has to be the current device."""
    if index != _current_device():
        raise ValueError(f"tensors are on cuda:{index}, the current device is "
                         f"cuda:{_current_device()}")
    raw = _raw_stream(index)
    if stream is None or stream.cuda_stream == raw:
        return raw, torch.empty
    return stream.cuda_stream, _Other(stream, index)


def _gpu(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    return t.get_device()


def _i32(t, index, name, shape):
    """Raise ValueError unless `t` is a contiguous int32 tensor of `shape` on GPU `index`."""
    if not (isinstance(t, torch.Tensor) and t.dtype is torch.int32 and t.get_device() == index and
            t.shape == shape and t.is_contiguous()):
        _check_dev(t, torch.device("cuda", index), name, torch.int32, shape, contiguous=True)


def _like(t, index, name, dtype, shape=None):
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index and
            (shape is None or t.shape == shape)):
        _check_dev(t, torch.device("cuda", index), name, dtype, shape)


def _pool(pool, index):
    """Entries of a pool of pages."""
    if not (isinstance(pool, torch.Tensor) and pool.dtype is torch.int32 and pool.dim() == 1 and
            pool.get_device() == index and pool.is_contiguous()):
        _gpu(pool, "pool")
        _check_dev(pool, torch.device("cuda", index), "pool", torch.int32, (pool.numel(),),
                   contiguous=True)
    return pool.shape[0]


def _tables(tables, index, rows):
    """(row stride, width) of page tables."""
    _like(tables, index, "tables", torch.int32)
    if tables.dim() == 2 and tables.shape[0] == rows:
        stride, one = tables.stride()
        width = tables.shape[1]
        if one == 1 or width <= 1:
            return (stride if rows > 1 else max(stride, width)), width
    raise ValueError("tables must be (rows, width) int32 with unit stride over the width")


def _cache(t, index, name, dtype, shape=None):
    _like(t, index, name, dtype, shape)
    if t.dim() == 4:
        page, token, head, one = t.stride()
        if one == 1 or t.shape[3] <= 1:
            return t.data_ptr(), page, token, head
    raise ValueError(f"{name} must be (pages, page_size, kv_heads, head_dim) with unit stride "
                     "over head_dim")


def _rows(t, name):
    """(row stride, head stride, shape) of a (rows, heads, head_dim) tensor."""
    if t.dim() == 3:
        row, head, one = t.stride()
        if one == 1 or t.shape[2] <= 1:
            return row, head, t.shape
    raise ValueError(f"{name} must have three axes, the last one with unit stride")


def _apart(t, strides, name):
    """Raise ValueError if elements of a tensor that is written share memory (an expanded
    axis): which of their values stays would be a matter of chance."""
    if 0 in strides and any(n > 1 and s == 0 for n, s in zip(t.shape, strides)):
        raise ValueError(f"{name} is written, and must not have expanded axes")


def _meet(a, b, d):
    """Whether two strided sets of bytes may share some.  a, b: (bytes from the first one to
    behind the last, item size, ((stride, count), ...) by descending stride); the second begins `d`
    behind the first.  False is certain."""
    if d >= a[0] or -d >= b[0]:
        return False
    if not a[2] or not b[2] or a[2][0][0] != b[2][0][0]:
        return True
    # both lie in strips `step` apart: a strip of the second beside each one of the first
    step = a[2][0][0]
    a, b = ((sum(s * (n - 1) for s, n in x[2][1:]) + x[1], x[1], x[2][1:]) for x in (a, b))
    if a[0] > step or b[0] > step:
        return True
    return _meet(a, b, d % step) or _meet(a, b, d % step - step)


def _off(out, t, name):
    """Raise ValueError if `out`, which is written, may overlap the input `t`: what a part of the
    kernel has written, another would read."""
    if not out.numel() or not t.numel():
        return
    sets = []
    for x in (out, t):
        axes = sorted(((s * x.itemsize, n) for s, n in zip(x.stride(), x.shape) if s and n > 1),
                      reverse=True)
        sets.append((sum(s * (n - 1) for s, n in axes) + x.itemsize, x.itemsize, axes))
    if _meet(*sets, t.data_ptr() - out.data_ptr()):
        raise ValueError(f"out must not overlap {name}")


def _type(t, name):
    dt = _TYPES.get(t.dtype)
    if dt is None:
        raise ValueError(f"{name} must be bfloat16, float16 or float32, got {t.dtype}")
    return dt


class CachePlan(NamedTuple):
    """What ``cache_plan`` made of a step: all int32 on the GPU."""
    slots: torch.Tensor       # (total,) slot of each new token, -1 without one
    positions: torch.Tensor   # (total,) its position in its request
    starts: torch.Tensor      # (rows + 1,) where each request's new tokens begin
    lengths: torch.Tensor     # (rows,) tokens held afterwards
    taken: torch.Tensor       # (1,) pool entries in use afterwards
    status: torch.Tensor      # (rows,) NO_PAGE | NO_ENTRY | NO_SLOT, 0 = complete


def cache_plan(lengths, counts, tables, pool, taken, page_size: int, total: int,
               stream=None) -> CachePlan:
    """Hand out pages for counts[r] new tokens of every request that already
    holds lengths[r] and list their slots.  `tables` (rows, width) gets the new
    pages' entries; pages come from pool[taken] on.  `total` is the size of the
    slot map: tokens past it are not appended.  All tensors int32 on the GPU;
    no input but `tables` changes, so the call can be repeated."""
    dev = _gpu(lengths, "lengths")
    rows = lengths.numel()
    _i32(lengths, dev, "lengths", (rows,))
    _i32(counts, dev, "counts", (rows,))
    stride, width = _tables(tables, dev, rows)
    pages = _pool(pool, dev)
    _i32(taken, dev, "taken", (1,))
    if not 0 <= total <= 1 << 30:
        raise ValueError("total must be in 0 .. 2^30")
    raw, empty = _on(stream, dev)
    # one allocation for all outputs
    buf = empty((2 * total + 3 * rows + 2,), dtype=torch.int32, device=lengths.device)
    base = buf.data_ptr()
    at = base + 8 * total
    _check(lib().ctcpb_lm_cache_plan(_pack(
        _PLAN, lengths.data_ptr(), counts.data_ptr(), tables.data_ptr(), pool.data_ptr(),
        taken.data_ptr(), base, base + 4 * total, at, at + 4 * (rows + 1),
        at + 4 * (2 * rows + 1), at + 4 * (2 * rows + 2), stride, rows, width, pages, page_size,
        total), raw))
    return CachePlan._make(buf.split_with_sizes((total, total, rows + 1, rows, 1, rows)))


def cache_release(finished, lengths, tables, pool, taken, page_size: int, stream=None):
    """Give the pages of the requests with finished[r] != 0 (uint8 or bool on the GPU)
    back to the pool.  Returns (lengths, taken) afterwards; `pool` changes below
    `taken` only, so the call can be repeated on the same inputs."""
    dev = _gpu(lengths, "lengths")
    rows = lengths.numel()
    if isinstance(finished, torch.Tensor) and finished.dtype == torch.bool:
        finished = finished.view(torch.uint8)
    _check_dev(finished, lengths.device, "finished", torch.uint8, (rows,), contiguous=True)
    _i32(lengths, dev, "lengths", (rows,))
    stride, width = _tables(tables, dev, rows)
    pages = _pool(pool, dev)
    _i32(taken, dev, "taken", (1,))
    raw, empty = _on(stream, dev)
    buf = empty((rows + 1,), dtype=torch.int32, device=lengths.device)
    base = buf.data_ptr()
    _check(lib().ctcpb_lm_cache_release(_pack(
        _RELEASE, finished.data_ptr(), lengths.data_ptr(), tables.data_ptr(), pool.data_ptr(),
        taken.data_ptr(), base, base + 4 * rows, stride, rows, width, pages, page_size), raw))
    return buf[:rows], buf[rows:]


def cache_store(k, v, slots, k_cache, v_cache, stream=None):
    """Write keys and values k, v (tokens, kv_heads, head_dim) to their slots
    (int32 (tokens,), distinct; -1 leaves a token out) of the caches (pages,
    page_size, kv_heads, head_dim), whose axes may lie in any order in memory
    with head_dim innermost."""
    dev = _gpu(k, "k")
    dt = _type(k, "k")
    kt, kh, shape = _rows(k, "k")
    _like(v, dev, "v", k.dtype, shape)
    vt, vh, _ = _rows(v, "v")
    T, H, D = shape
    _i32(slots, dev, "slots", (T,))
    kc = _cache(k_cache, dev, "k_cache", k.dtype)
    pages, page_size, heads, dim = cs = k_cache.shape
    vc = _cache(v_cache, dev, "v_cache", k.dtype, cs)
    _apart(k_cache, kc[1:], "k_cache")
    _apart(v_cache, vc[1:], "v_cache")
    if heads != H or dim != D:
        raise ValueError(f"caches must have {H} heads of {D}, got {(heads, dim)}")
    if T == 0:
        return
    _check(lib().ctcpb_lm_cache_store(_pack(
        _STORE, k.data_ptr(), v.data_ptr(), slots.data_ptr(), kt, kh, vt, vh, *kc, *vc, dt, T,
        pages, page_size, H, D), _on(stream, dev)[0]))


def attention(q, k_cache, v_cache, tables, lengths, scale: float | None = None, window: int = 0,
              max_len: int = 0, out=None, stream=None):
    """Attention of one token per request over its pages: q (rows, q_heads,
    head_dim), caches (pages, page_size, kv_heads, head_dim), tables (rows,
    width) and lengths (rows,) int32 as ``cache_plan`` leaves them, the new
    token stored.  `window` > 0 keeps the last `window` tokens only; `max_len` is an
    upper bound of the lengths, where the caller knows a closer one than the
    tables' width.  Returns (out like q, lse (rows, q_heads) float32); a request
    without tokens gives zeros and -inf."""
    dev = _gpu(q, "q")
    dt = _type(q, "q")
    qr, qh, shape = _rows(q, "q")
    R, Hq, D = shape
    kc = _cache(k_cache, dev, "k_cache", q.dtype)
    pages, page_size, Hkv, Dk = cs = k_cache.shape
    vc = _cache(v_cache, dev, "v_cache", q.dtype, cs)
    if Dk != D:
        raise ValueError(f"caches must have heads of {D}, got {Dk}")
    stride, width = _tables(tables, dev, R)
    _i32(lengths, dev, "lengths", (R,))
    L = lib()
    raw, empty = _on(stream, dev)
    if out is None:
        out = empty(shape, dtype=q.dtype, device=q.device)
    else:
        _like(out, dev, "out", q.dtype, shape)
    outr, outh, _ = _rows(out, "out")
    _apart(out, (outr, outh), "out")
    lse = empty((R, Hq), dtype=torch.float32, device=q.device)
    args = _pack(
        _ATTENTION, q.data_ptr(), tables.data_ptr(), lengths.data_ptr(), out.data_ptr(),
        lse.data_ptr(), qr, qh, outr, outh, stride, *kc, *vc, dt, R, Hq, Hkv, D, pages, page_size,
        width, max_len, window, 1.0 / math.sqrt(D) if scale is None else scale)
    need = ctypes.c_size_t()
    _check(L.ctcpb_lm_attention_workspace(args, need))
    size = need.value
    # freed on return: the stream's later work may have it, after this call
    ws = empty((size,), dtype=torch.uint8, device=q.device) if size else None
    _check(L.ctcpb_lm_attention(args, ws.data_ptr() if size else None, size, raw))
    return out, lse


def _loss_args(x, w, targets, bias):
    dev = _gpu(x, "x")
    dt = _type(x, "x")
    if x.dim() != 2 or (x.stride(1) != 1 and x.shape[1] > 1):
        raise ValueError("x must be (rows, hidden) with unit stride over hidden")
    N, H = x.shape
    _like(w, dev, "w", x.dtype)
    if w.dim() != 2 or w.shape[1] != H or (w.stride(1) != 1 and H > 1):
        raise ValueError(f"w must be (vocab, {H}) with unit stride over hidden")
    V = w.shape[0]
    _i32(targets, dev, "targets", (N,))
    if bias is not None:
        _floats(bias, dev, "bias", V)
    # a single row's stride is of no account, and may be anything
    sx = x.stride(0) if N > 1 else H
    sw = w.stride(0) if V > 1 else H
    return dev, N, V, H, (sx, sw, dt, N, V, H)


def _floats(t, index, name, n):
    _like(t, index, name, torch.float32, (n,))
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def token_loss_forward(x, w, targets, bias=None, stream=None):
    """(loss, lse), both (rows,) float32, of an output layer: x (rows, hidden), w
    (vocab, hidden) of one type, bias float32 (vocab,) or None, targets int32
    (rows,).  loss = lse - logit of the target, 0 where the target is outside
    the vocabulary (the decoder's -1 padding)."""
    dev, N, V, H, sizes = _loss_args(x, w, targets, bias)
    L = lib()
    raw, empty = _on(stream, dev)
    loss = empty((N,), dtype=torch.float32, device=x.device)
    lse = empty((N,), dtype=torch.float32, device=x.device)
    args = _pack(_LOSS, x.data_ptr(), w.data_ptr(), _ptr(bias), targets.data_ptr(),
                 loss.data_ptr(), lse.data_ptr(), *sizes)
    need = ctypes.c_size_t()
    _check(L.ctcpb_lm_loss_workspace(args, need))
    ws = empty((need.value,), dtype=torch.uint8, device=x.device)
    _check(L.ctcpb_lm_loss(args, ws.data_ptr(), need.value, raw))
    return loss, lse


def token_loss_backward(grad, x, w, targets, lse, bias=None, need=(True, True, True), stream=None,
                        split_d: bool = False):
    """Gradients (dx, dw, dbias) of sum(grad * loss) for ``token_loss_forward``
    with its lse; grad (rows,) float32.  dx and dw have x's and w's type, dbias
    is float32 (None without a bias).  `need` says which of them to compute.  Rows
    whose target is outside the vocabulary add nothing (for dw their x has to be finite).

    With 16-bit types the gradients of the logits are rounded to that type on the
    way: the errors of dx and dw are mostly 1.0 to 1.4 times those of rounding the exact
    results, up to 2.2 times where most rows share a weight that is not the largest.
    `split_d` keeps them as the sum of two such values (as is done in small calls
    anyway), which leaves the results' own rounding, at twice the products."""
    dev, N, V, H, sizes = _loss_args(x, w, targets, bias)
    if split_d:
        sizes = sizes[:2] + (sizes[2] | _SPLIT_D,) + sizes[3:]
    _floats(grad, dev, "grad", N)
    _floats(lse, dev, "lse", N)
    L = lib()
    raw, empty = _on(stream, dev)
    dx = empty((N, H), dtype=x.dtype, device=x.device) if need[0] else None
    dw = empty((V, H), dtype=w.dtype, device=x.device) if need[1] else None
    db = None
    if need[2] and bias is not None:
        db = empty((V,), dtype=torch.float32, device=x.device)
    args = _pack(_GRAD, x.data_ptr(), w.data_ptr(), _ptr(bias), targets.data_ptr(),
                 grad.data_ptr(), lse.data_ptr(), _ptr(dx), _ptr(dw), _ptr(db), *sizes)
    size = ctypes.c_size_t()
    _check(L.ctcpb_lm_loss_grad_workspace(args, size))
    ws = empty((size.value,), dtype=torch.uint8, device=x.device)
    _check(L.ctcpb_lm_loss_grad(args, ws.data_ptr(), size.value, raw))
    return dx, dw, db


class _TokenLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, targets, bias, split_d):
        loss, lse = token_loss_forward(x, w, targets, bias)
        ctx.split_d = split_d
        ctx.save_for_backward(x, w, targets, bias, lse)
        return loss

    @staticmethod
    def backward(ctx, grad):
        x, w, targets, bias, lse = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dw, db = token_loss_backward(grad.contiguous(), x, w, targets, lse, bias,
                                         (need[0], need[1], need[3]), split_d=ctx.split_d)
        if torch.is_grad_enabled():   # create_graph: the gradients are asked to have a graph
            dx, dw, db = _Last.apply((dx, dw, db), grad, x, w, bias)
        return dx, dw, None, db, None


class _Last(torch.autograd.Function):
    """Gradients that cannot be differentiated again: the library's carry no graph, and what
    would follow from them would be left out without a word."""

    @staticmethod
    def forward(ctx, gradients, *of):
        return tuple(None if g is None else g.view_as(g) for g in gradients)

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("token_loss cannot be differentiated twice")


def token_loss(x, w, targets, bias=None, split_d: bool = False):
    """The losses of ``token_loss_forward`` as a torch function: gradients flow
    to x, w and bias (`split_d`: see ``token_loss_backward``).  First derivatives
    only; differentiating them again raises."""
    return _TokenLoss.apply(x, w, targets, bias, split_d)


def _codes(t, name):
    code = _CODES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be int8 or float8_e4m3fn, got {t.dtype}")
    return code


def _cache8(k_cache, v_cache, k_scale, v_scale, index, written, caller):
    """(code, (pages, page_size, heads, dim), the caches' and scales' addresses and strides)."""
    _gpu(k_cache, "k_cache")
    dtype = k_cache.dtype
    code = _codes(k_cache, "k_cache")
    kc = _cache(k_cache, index, "k_cache", dtype)
    shape = k_cache.shape
    vc = _cache(v_cache, index, "v_cache", dtype, shape)
    each = (shape[0], shape[2])
    _like(k_scale, index, "k_scale", torch.float32, each)
    _like(v_scale, index, "v_scale", torch.float32, each)
    if (k_cache.requires_grad or v_cache.requires_grad or k_scale.requires_grad or
            v_scale.requires_grad):
        _no_gradient(caller)
    ks, vs = k_scale.stride(), v_scale.stride()
    if written:
        _apart(k_cache, kc[1:], "k_cache")
        _apart(v_cache, vc[1:], "v_cache")
        _apart(k_scale, ks, "k_scale")
        _apart(v_scale, vs, "v_scale")
    return code, shape, kc + vc, (k_scale.data_ptr(), *ks, v_scale.data_ptr(), *vs)


def _no_gradient(name):
    """Raise ValueError for a call with tensors that ask for gradients, which it cannot give."""
    if torch.is_grad_enabled():
        raise ValueError(f"{name} carries no gradients: call it under torch.no_grad() or on "
                         "detached tensors")


def cache_store8(k, v, slots, k_cache, v_cache, k_scale, v_scale, stream=None):
    """``cache_store`` to caches of 8-bit codes (int8 or float8_e4m3fn, (pages, page_size,
    kv_heads, head_dim)) with float32 scales (pages, kv_heads).  A page's scale is the least
    power of two with which the largest code (127 or 448) reaches all that was written to it; it
    starts with the token of slot 0, which begins the page anew, and later tokens can only raise
    it: what the page holds is then rescaled.  Slots are distinct, 2^30 at most, and the tokens of
    a page follow one another, as ``cache_plan`` lays them out (``cache_store`` takes any order).
    Values are at most half a step off, rescaled ones less than one; one that is not finite makes
    its page's scale NaN, until the page begins anew."""
    dev = _gpu(k, "k")
    dt = _type(k, "k")
    kt, kh, shape = _rows(k, "k")
    _like(v, dev, "v", k.dtype, shape)
    if k.requires_grad or v.requires_grad:
        _no_gradient("cache_store8")
    vt, vh, _ = _rows(v, "v")
    T, H, D = shape
    _i32(slots, dev, "slots", (T,))
    code, (pages, page_size, heads, dim), caches, scales = _cache8(
        k_cache, v_cache, k_scale, v_scale, dev, True, "cache_store8")
    if heads != H or dim != D:
        raise ValueError(f"caches must have {H} heads of {D}, got {(heads, dim)}")
    if T == 0:
        return
    _check(lib().ctcpb_lm_cache_store8(_pack(
        _CACHE8, k.data_ptr(), v.data_ptr(), slots.data_ptr(), kt, kh, vt, vh, *caches, *scales, dt,
        code, T, pages, page_size, H, D), _on(stream, dev)[0]))


def cache_load8(slots, k_cache, v_cache, k_scale, v_scale, dtype=torch.bfloat16, stream=None):
    """(k, v), both (tokens, kv_heads, head_dim) of `dtype`: what the slots (int32 (tokens,)) of
    an 8-bit cache hold, code times scale, as the largest value of `dtype` where a finite product
    is past it; zeros for a token without a slot (-1)."""
    dev = _gpu(slots, "slots")
    T = slots.numel()
    _i32(slots, dev, "slots", (T,))
    dt = _TYPES.get(dtype)
    if dt is None:
        raise ValueError(f"dtype must be bfloat16, float16 or float32, got {dtype}")
    code, (pages, page_size, H, D), caches, scales = _cache8(
        k_cache, v_cache, k_scale, v_scale, dev, False, "cache_load8")
    raw, empty = _on(stream, dev)
    both = empty((2, T, H, D), dtype=dtype, device=slots.device)
    at = both.data_ptr()
    _check(lib().ctcpb_lm_cache_load8(_pack(
        _CACHE8, at, at + T * H * D * dtype.itemsize, slots.data_ptr(), H * D, D, H * D, D, *caches,
        *scales, dt, code, T, pages, page_size, H, D), raw))
    return both.unbind(0)


def attention8(q, k_cache, v_cache, k_scale, v_scale, tables, lengths, scale: float | None = None,
               window: int = 0, max_len: int = 0, out=None, stream=None):
    """``attention`` over caches of 8-bit codes (int8 or float8_e4m3fn) with float32 scales
    (pages, kv_heads) >= 0: keys and values are code times scale of their page and head.  q and
    out are bfloat16, float16 or float32 (finite results past float16's end become its largest
    value); head_dim is a multiple of 16.  `out` may be q."""
    dev = _gpu(q, "q")
    if q.requires_grad:
        _no_gradient("attention8")
    dt = _type(q, "q")
    qr, qh, shape = _rows(q, "q")
    R, Hq, D = shape
    code, (pages, page_size, Hkv, Dk), caches, scales = _cache8(
        k_cache, v_cache, k_scale, v_scale, dev, False, "attention8")
    if Dk != D:
        raise ValueError(f"caches must have heads of {D}, got {Dk}")
    stride, width = _tables(tables, dev, R)
    _i32(lengths, dev, "lengths", (R,))
    L = lib()
    raw, empty = _on(stream, dev)
    if out is None:
        out = empty(shape, dtype=q.dtype, device=q.device)
    else:
        _like(out, dev, "out", q.dtype, shape)
        if out.requires_grad:
            _no_gradient("attention8")
        if out.data_ptr() != q.data_ptr() or out.stride() != q.stride():
            _off(out, q, "q")
    outr, outh, _ = _rows(out, "out")
    _apart(out, (outr, outh), "out")
    lse = empty((R, Hq), dtype=torch.float32, device=q.device)
    args = _pack(
        _ATTENTION8, q.data_ptr(), tables.data_ptr(), lengths.data_ptr(), out.data_ptr(),
        lse.data_ptr(), qr, qh, outr, outh, stride, *caches, dt, R, Hq, Hkv, D, pages, page_size,
        width, max_len, window, 1.0 / math.sqrt(D) if scale is None else scale, *scales, code)
    need = ctypes.c_size_t()
    _check(L.ctcpb_lm_attention8_workspace(args, need))
    size = need.value
    # freed on return: the stream's later work may have it, after this call
    ws = empty((size,), dtype=torch.uint8, device=q.device) if size else None
    _check(L.ctcpb_lm_attention8(args, ws.data_ptr() if size else None, size, raw))
    return out, lse


def _matrix(t, name, columns=None):
    """(row stride, rows, columns) of a matrix with unit stride over its columns."""
    if t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] > 1):
        raise ValueError(f"{name} must have two axes, the last one with unit stride")
    rows, n = t.shape
    if columns is not None and n != columns:
        raise ValueError(f"{name} must have {columns} columns, got {n}")
    # a single row's stride is of no account, and may be anything
    return (t.stride(0) if rows > 1 else n), rows, n


def quantize_rows(x, stream=None):
    """(codes, scales) of the rows of x (rows, hidden): codes int8 (rows, hidden), x = codes *
    scales[:, None] up to half a step, scales float32 (rows,) = max |x| / 127 of each row.  A row
    with a value that is not finite has the scale NaN.  Rows of codes begin on 16 bytes, with
    zeros behind them, as ``linear8`` reads them best."""
    dev = _gpu(x, "x")
    if x.requires_grad:
        _no_gradient("quantize_rows")
    dt = _type(x, "x")
    sx, N, H = _matrix(x, "x")
    if H == 0:
        raise ValueError("x must have columns")
    raw, empty = _on(stream, dev)
    wide = -(-H // 16) * 16
    codes = empty((N, wide), dtype=torch.int8, device=x.device)
    scales = empty((N,), dtype=torch.float32, device=x.device)
    _check(lib().ctcpb_lm_quantize_rows(_pack(
        _QUANTIZE, x.data_ptr(), codes.data_ptr(), scales.data_ptr(), sx, wide, dt, N, H), raw))
    return (codes if wide == H else codes[:, :H]), scales


def _readable(t, stride, rows, columns):
    """Whether the last row of codes, too, can be read up to the next multiple of 16."""
    wide = -(-columns // 16) * 16
    return (wide == columns or
            t.storage_offset() + (rows - 1) * stride + wide <= t.untyped_storage().nbytes())


def linear8(x, w, w_scale, bias=None, x_scale=None, dtype=None, out=None, stream=None):
    """x times 8-bit weights: (sum over hidden of codes) * x_scale * w_scale + bias, (rows,
    features).  w int8 (features, hidden) with w_scale float32 (features,), as
    ``quantize_rows`` makes them of a weight.  x (rows, hidden) is either bfloat16, float16
    or float32, and quantised by row on the way (out then has its type), or int8 codes with their
    x_scale float32 (rows,), and `dtype` (default bfloat16) is that of out.  bias: float32
    (features,) or None.  Sums of codes are exact; hidden is at most 131071."""
    dev = _gpu(x, "x")
    sx, N, H = _matrix(x, "x")
    _like(w, dev, "w", torch.int8)
    sw, M, _ = _matrix(w, "w", H)
    _floats(w_scale, dev, "w_scale", M)
    if bias is not None:
        _floats(bias, dev, "bias", M)
    if x.requires_grad or w_scale.requires_grad or (bias is not None and bias.requires_grad):
        _no_gradient("linear8")
    flags = _READABLE if _readable(w, sw, M, H) else 0
    if x.dtype is torch.int8:
        if x_scale is None:
            raise ValueError("x of int8 codes needs x_scale")
        _floats(x_scale, dev, "x_scale", N)
        if x_scale.requires_grad:
            _no_gradient("linear8")
        xt, dtype = _CODES_X, dtype or torch.bfloat16
    else:
        if x_scale is not None:
            raise ValueError("x_scale is for x of int8 codes")
        xt = _type(x, "x")
        if dtype not in (None, x.dtype):
            raise ValueError(f"out has x's type, {x.dtype}; dtype is for x of int8 codes")
        dtype = x.dtype
    dt = _TYPES.get(dtype)
    if dt is None:
        raise ValueError(f"dtype must be bfloat16, float16 or float32, got {dtype}")
    L = lib()
    raw, empty = _on(stream, dev)
    if out is None:
        out = empty((N, M), dtype=dtype, device=x.device)
    else:
        _like(out, dev, "out", dtype, (N, M))
        if out.requires_grad:
            _no_gradient("linear8")
        for t, name in ((x, "x"), (w, "w"), (w_scale, "w_scale"), (bias, "bias"),
                        (x_scale, "x_scale")):
            if t is not None:
                _off(out, t, name)
    so, _, _ = _matrix(out, "out")
    _apart(out, out.stride(), "out")
    args = _pack(_LINEAR8, x.data_ptr(), _ptr(x_scale), w.data_ptr(), w_scale.data_ptr(),
                 _ptr(bias), out.data_ptr(), sx, sw, so, xt, dt, N, M, H, flags)
    need = ctypes.c_size_t()
    _check(L.ctcpb_lm_linear8_workspace(args, need))
    size = need.value
    ws = empty((size,), dtype=torch.uint8, device=x.device) if size else None
    _check(L.ctcpb_lm_linear8(args, ws.data_ptr() if size else None, size, raw))
    return out


class PagedCache:
    """The paged key/value cache of a model's attention layers and its page
    allocator, for `rows` requests of at most `max_len` tokens each, rounded up to
    whole pages (`self.max_len`): tokens past that have no slot, and are flagged.
    The layers share their pages' numbers, so one plan serves them all.

    ``append(counts, total)`` hands out pages, ``store(k, v, slots, layer)``
    writes a layer's new tokens, ``attend(q, layer)`` attends over each request's
    tokens (`max_len`: a closer bound of the lengths, where the caller knows one), and
    ``release(finished)`` gives pages back.  `num_pages` (default:
    every request at max_len) may be smaller: a request the pool cannot serve is
    flagged in the plan's status and holds only the tokens that have a slot.  Use
    one PagedCache per stream, or order its calls.

    With `dtype` int8 or float8_e4m3fn (head_dim a multiple of 16) the cache holds codes, and
    ``k_scale`` and ``v_scale`` (layers, num_pages, kv_heads) their scales: ``store`` quantises
    (``cache_store8``), ``attend`` is ``attention8``, and ``load(slots, layer)`` reads tokens back
    in 16 or 32 bits.  A page's tokens share a scale, so ``store`` then needs what ``append`` gives:
    the tokens of a page one after another in the call.  (In 16 and 32 bits tokens may come in any
    order.)  Tokens of a page with those of another one between them would be done at the same
    time, and leave the page with either scale and codes of both.

    An append goes on to the plan's new lengths, so a captured one repeats the same
    step when it is replayed.  To capture a step that moves on, call ``cache_plan``
    and copy its lengths and `taken` back to the tensors that it reads."""

    def __init__(self, rows: int, max_len: int, kv_heads: int, head_dim: int,
                 dtype=torch.bfloat16, page_size: int = 16, num_pages: int = 0, device="cuda",
                 layers: int = 1):
        if page_size not in (4, 8, 16, 32, 64, 128, 256):
            raise ValueError("page_size must be a power of two in 4..256")
        if min(rows, max_len, num_pages) < 0:
            raise ValueError("rows, max_len and num_pages must be >= 0")
        if dtype in _CODES and (head_dim % 16 or not 0 < head_dim <= 256):   # what attend takes
            raise ValueError("head_dim must be a multiple of 16 up to 256 with a dtype of codes, "
                             f"got {head_dim}")
        width = -(-max_len // page_size)
        num_pages = num_pages or max(1, rows * width)
        self.page_size, self.max_len = page_size, width * page_size
        self.k_scale = self.v_scale = None
        if dtype in _CODES:
            # head by head: rows are short, and a page's of one head then lie together, as do
            # its two scales
            both = [torch.empty((layers, num_pages, kv_heads, page_size, head_dim), dtype=dtype,
                                device=device).transpose(2, 3) for _ in range(2)]
            self.k, self.v = both
            scales = torch.zeros((layers, num_pages, kv_heads, 2), device=device)
            self.k_scale, self.v_scale = scales.unbind(-1)
        else:
            self.k = torch.empty((layers, num_pages, page_size, kv_heads, head_dim), dtype=dtype,
                                 device=device)
            self.v = torch.empty_like(self.k)
        self.tables = torch.full((rows, width), -1, dtype=torch.int32, device=device)
        self.pool = torch.arange(num_pages, dtype=torch.int32, device=device)
        self.lengths = torch.zeros(rows, dtype=torch.int32, device=device)
        self.taken = torch.zeros(1, dtype=torch.int32, device=device)

    def _keep(self, stream, *tensors):
        """Marks `tensors` as used by the call just made on `stream` (None: the current
        one), so that their memory, should the cache give it up, is not handed out again
        before that call has run: it may belong to another stream."""
        if stream is None:
            stream = torch.cuda.current_stream(self.k.device)
        for t in tensors:
            t.record_stream(stream)

    def append(self, counts, total: int, stream=None) -> CachePlan:
        plan = cache_plan(self.lengths, counts, self.tables, self.pool, self.taken,
                          self.page_size, total, stream)
        self._keep(stream, self.lengths, self.taken, self.tables, self.pool)
        self.lengths, self.taken = plan.lengths, plan.taken
        return plan

    def _codes(self, layer):
        """A layer's codes and scales."""
        return self.k[layer], self.v[layer], self.k_scale[layer], self.v_scale[layer]

    def store(self, k, v, slots, layer: int = 0, stream=None):
        if self.k_scale is None:
            cache_store(k, v, slots, self.k[layer], self.v[layer], stream)
            self._keep(stream, self.k, self.v)
        else:
            cache_store8(k, v, slots, *self._codes(layer), stream)
            self._keep(stream, self.k, self.v, self.k_scale, self.v_scale)

    def load(self, slots, layer: int = 0, dtype=torch.bfloat16, stream=None):
        """(k, v) of the tokens in `slots`, of an 8-bit cache."""
        if self.k_scale is None:
            raise ValueError("load is for caches of int8 or float8_e4m3fn")
        got = cache_load8(slots, *self._codes(layer), dtype, stream)
        self._keep(stream, self.k, self.v, self.k_scale, self.v_scale)
        return got

    def attend(self, q, layer: int = 0, scale=None, window: int = 0, max_len: int = 0, stream=None):
        if self.k_scale is None:
            got = attention(q, self.k[layer], self.v[layer], self.tables, self.lengths, scale,
                            window, max_len, stream=stream)
            self._keep(stream, self.k, self.v, self.tables, self.lengths)
        else:
            got = attention8(q, *self._codes(layer), self.tables, self.lengths, scale, window,
                             max_len, stream=stream)
            self._keep(stream, self.k, self.v, self.k_scale, self.v_scale, self.tables,
                       self.lengths)
        return got

    def release(self, finished, stream=None):
        lengths, taken = cache_release(finished, self.lengths, self.tables, self.pool, self.taken,
                                       self.page_size, stream)
        self._keep(stream, self.lengths, self.taken, self.tables, self.pool)
        self.lengths, self.taken = lengths, taken
