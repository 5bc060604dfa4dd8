"""Operators for rescoring N-best lists with a language model on MI355X.

Thin Python binding of ``libctcpb_lm.so`` (C ABI in ``include/ctcpb_lm.h``):
the pages and slots of a paged key/value cache from device-resident lengths
(``cache_plan``, ``cache_release``), the store of new tokens' keys and values
(``cache_store``), the attention of one new token per request over the cache
(``attention``), and token losses over a large vocabulary without keeping the
logits, with their gradients (``token_loss``).  ``PagedCache`` holds the tensors
of a cache.  Every step
runs in the library's HIP kernels; PyTorch provides device memory and the
current stream.  If the library is missing the calls raise; there is no CPU
fallback.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import NamedTuple

import torch

from . import _check_dev

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libctcpb_lm.so")

EXPORTS = ("ctcpb_lm_cache_plan", "ctcpb_lm_cache_release", "ctcpb_lm_cache_store",
           "ctcpb_lm_attention_workspace", "ctcpb_lm_attention", "ctcpb_lm_loss_workspace",
           "ctcpb_lm_loss", "ctcpb_lm_loss_grad_workspace", "ctcpb_lm_loss_grad",
           "ctcpb_lm_last_error")
NO_PAGE, NO_ENTRY, NO_SLOT = 1, 2, 4   # status bits of cache_plan
_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


class CtcpbLmCache(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride_page", ctypes.c_int64),
                ("stride_token", ctypes.c_int64), ("stride_head", ctypes.c_int64)]


_lib = None


def lib():
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with ctc_prefix_beam_amd.build")
        L = ctypes.CDLL(LIB_PATH)
        p, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        f32, cachep, szp = ctypes.c_float, ctypes.POINTER(CtcpbLmCache), ctypes.POINTER(sz)
        L.ctcpb_lm_cache_plan.argtypes = [p, p, i32, p, i64, i32, p, i32, p, i32, p, p, i32, p, p,
                                          p, p, p]
        L.ctcpb_lm_cache_release.argtypes = [p, p, i32, p, i64, i32, p, i32, p, i32, p, p, p]
        L.ctcpb_lm_cache_store.argtypes = [i32, p, i64, i64, p, i64, i64, p, i32, cachep, cachep,
                                           i32, i32, i32, i32, p]
        L.ctcpb_lm_attention_workspace.argtypes = [i32, i32, i32, i32, i32, i32, i32, szp]
        L.ctcpb_lm_attention.argtypes = [i32, p, i64, i64, cachep, cachep, i32, i32, p, i64, i32,
                                         p, i32, i32, i32, i32, i32, i32, f32, p, i64, i64, p, p,
                                         sz, p]
        L.ctcpb_lm_loss_workspace.argtypes = [i32, p, i64, p, i64, i32, i32, i32, szp]
        L.ctcpb_lm_loss.argtypes = [i32, p, i64, p, i64, p, p, i32, i32, i32, p, p, p, sz, p]
        L.ctcpb_lm_loss_grad_workspace.argtypes = [i32, p, i64, p, i64, i32, i32, i32, szp]
        L.ctcpb_lm_loss_grad.argtypes = [i32, p, p, i64, p, i64, p, p, p, i32, i32, i32, p, p, p,
                                         p, sz, p]
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


class _On:
    """The stream a call runs on, and the memory it allocates for itself: made
    on the current stream, and marked as used by `stream` if that is another
    one, so that it is not handed out again while the call still runs."""

    def __init__(self, stream, device):
        if device.index != torch.cuda.current_device():
            raise ValueError(f"tensors are on {device}, which is not the current device "
                             f"({torch.cuda.current_device()})")
        self.current = torch.cuda.current_stream(device)
        self.stream = self.current if stream is None else stream
        self.other = self.stream.cuda_stream != self.current.cuda_stream
        self.device = device
        self.ptr = self.stream.cuda_stream

    def empty(self, shape, dtype):
        t = torch.empty(shape, dtype=dtype, device=self.device)
        if self.other:
            # it may have been in use on the current stream until now
            self.stream.wait_stream(self.current)
            t.record_stream(self.stream)
        return t


def _gpu(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    return t.device


def _i32(t, device, name, shape):
    _check_dev(t, device, name, torch.int32, shape, contiguous=True)


def _tables(tables, device, rows):
    _check_dev(tables, device, "tables", torch.int32)
    if tables.dim() != 2 or tables.shape[0] != rows or (tables.shape[1] > 1 and
                                                        tables.stride(1) != 1):
        raise ValueError("tables must be (rows, width) int32 with unit stride over the width")
    return max(tables.stride(0), tables.shape[1]) if rows <= 1 else tables.stride(0)


def _cache(t, device, name, dtype, shape=None):
    _check_dev(t, device, name, dtype, shape)
    if t.dim() != 4 or (t.shape[3] > 1 and t.stride(3) != 1):
        raise ValueError(f"{name} must be (pages, page_size, kv_heads, head_dim) with unit "
                         "stride over head_dim")
    return CtcpbLmCache(t.data_ptr(), t.stride(0), t.stride(1), t.stride(2))


def _type(t, name):
    if t.dtype not in _TYPES:
        raise ValueError(f"{name} must be bfloat16, float16 or float32, got {t.dtype}")
    return _TYPES[t.dtype]


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
    stride = _tables(tables, dev, rows)
    _i32(pool, dev, "pool", (pool.numel(),))
    _i32(taken, dev, "taken", (1,))
    if total < 0:
        raise ValueError("total must be >= 0")
    on = _On(stream, dev)
    # one allocation for all outputs
    buf = on.empty((2 * total + 3 * rows + 2,), torch.int32)
    slots, positions, starts, after, now, status = buf.split(
        (total, total, rows + 1, rows, 1, rows))
    base = buf.data_ptr()
    at = base + 8 * total
    _check(lib().ctcpb_lm_cache_plan(
        lengths.data_ptr(), counts.data_ptr(), rows, tables.data_ptr(), stride, tables.shape[1],
        pool.data_ptr(), pool.numel(), taken.data_ptr(), page_size, base, base + 4 * total, total,
        at, at + 4 * (rows + 1), at + 4 * (2 * rows + 1), at + 4 * (2 * rows + 2), on.ptr))
    return CachePlan(slots, positions, starts, after, now, status)


def cache_release(finished, lengths, tables, pool, taken, page_size: int, stream=None):
    """Give the pages of the requests with finished[r] != 0 (uint8 on the GPU)
    back to the pool.  Returns (lengths, taken) afterwards; `pool` changes below
    `taken` only, so the call can be repeated on the same inputs."""
    dev = _gpu(lengths, "lengths")
    rows = lengths.numel()
    _check_dev(finished, dev, "finished", torch.uint8, (rows,), contiguous=True)
    _i32(lengths, dev, "lengths", (rows,))
    stride = _tables(tables, dev, rows)
    _i32(pool, dev, "pool", (pool.numel(),))
    _i32(taken, dev, "taken", (1,))
    on = _On(stream, dev)
    buf = on.empty((rows + 1,), torch.int32)
    base = buf.data_ptr()
    _check(lib().ctcpb_lm_cache_release(
        finished.data_ptr(), lengths.data_ptr(), rows, tables.data_ptr(), stride, tables.shape[1],
        pool.data_ptr(), pool.numel(), taken.data_ptr(), page_size, base, base + 4 * rows, on.ptr))
    return buf[:rows], buf[rows:]


def cache_store(k, v, slots, k_cache, v_cache, stream=None):
    """Write keys and values k, v (tokens, kv_heads, head_dim) to their slots
    (int32 (tokens,), distinct; -1 leaves a token out) of the caches (pages,
    page_size, kv_heads, head_dim), whose axes may lie in any order in memory
    with head_dim innermost."""
    dev = _gpu(k, "k")
    dt = _type(k, "k")
    if k.dim() != 3 or (k.shape[2] > 1 and k.stride(2) != 1):
        raise ValueError("k must be (tokens, kv_heads, head_dim) with unit stride over head_dim")
    T, H, D = k.shape
    _check_dev(v, dev, "v", k.dtype, (T, H, D))
    if D > 1 and v.stride(2) != 1:
        raise ValueError("v must have unit stride over head_dim")
    _i32(slots, dev, "slots", (T,))
    kc = _cache(k_cache, dev, "k_cache", k.dtype)
    vc = _cache(v_cache, dev, "v_cache", k.dtype, k_cache.shape)
    if tuple(k_cache.shape[2:]) != (H, D):
        raise ValueError(f"caches must have {H} heads of {D}, got {tuple(k_cache.shape[2:])}")
    if T == 0:
        return
    _check(lib().ctcpb_lm_cache_store(
        dt, k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(), v.stride(0), v.stride(1),
        slots.data_ptr(), T, ctypes.byref(kc), ctypes.byref(vc), k_cache.shape[0],
        k_cache.shape[1], H, D, _On(stream, dev).ptr))


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
    if q.dim() != 3 or (q.shape[2] > 1 and q.stride(2) != 1):
        raise ValueError("q must be (rows, q_heads, head_dim) with unit stride over head_dim")
    R, Hq, D = q.shape
    kc = _cache(k_cache, dev, "k_cache", q.dtype)
    vc = _cache(v_cache, dev, "v_cache", q.dtype, k_cache.shape)
    pages, page_size, Hkv, Dk = k_cache.shape
    if Dk != D:
        raise ValueError(f"caches must have heads of {D}, got {Dk}")
    stride = _tables(tables, dev, R)
    _i32(lengths, dev, "lengths", (R,))
    if out is not None:
        _check_dev(out, dev, "out", q.dtype, q.shape)
        if D > 1 and out.stride(2) != 1:
            raise ValueError("out must have unit stride over head_dim")
    L = lib()
    width = tables.shape[1]
    bound = width * page_size
    if 0 < max_len < bound:
        bound = max_len
    need = ctypes.c_size_t()
    _check(L.ctcpb_lm_attention_workspace(dt, R, Hq, Hkv, D, bound, window, ctypes.byref(need)))
    on = _On(stream, dev)
    if out is None:
        out = on.empty((R, Hq, D), q.dtype)
    lse = on.empty((R, Hq), torch.float32)
    ws = on.empty((need.value,), torch.uint8) if need.value else None
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    _check(L.ctcpb_lm_attention(
        dt, q.data_ptr(), q.stride(0), q.stride(1), ctypes.byref(kc), ctypes.byref(vc), pages,
        page_size, tables.data_ptr(), stride, width, lengths.data_ptr(), R, Hq, Hkv, D, bound,
        window, scale, out.data_ptr(), out.stride(0), out.stride(1), lse.data_ptr(),
        ws.data_ptr() if ws is not None else None, need.value, on.ptr))
    return out, lse


def _loss_args(x, w, targets, bias):
    dev = _gpu(x, "x")
    dt = _type(x, "x")
    if x.dim() != 2 or (x.shape[1] > 1 and x.stride(1) != 1):
        raise ValueError("x must be (rows, hidden) with unit stride over hidden")
    N, H = x.shape
    _check_dev(w, dev, "w", x.dtype)
    if w.dim() != 2 or w.shape[1] != H or (H > 1 and w.stride(1) != 1):
        raise ValueError(f"w must be (vocab, {H}) with unit stride over hidden")
    V = w.shape[0]
    _i32(targets, dev, "targets", (N,))
    if bias is not None:
        _check_dev(bias, dev, "bias", torch.float32, (V,), contiguous=True)
    # a single row's stride is of no account, and may be anything
    sx = x.stride(0) if N > 1 else H
    sw = w.stride(0) if V > 1 else H
    return dev, dt, N, V, H, sx, sw


def _ptr(t):
    return t.data_ptr() if t is not None else None


def token_loss_forward(x, w, targets, bias=None, stream=None):
    """(loss, lse), both (rows,) float32, of an output layer: x (rows, hidden), w
    (vocab, hidden) of one type, bias float32 (vocab,) or None, targets int32
    (rows,).  loss = lse - logit of the target, 0 where the target is outside
    the vocabulary (the decoder's -1 padding)."""
    dev, dt, N, V, H, sx, sw = _loss_args(x, w, targets, bias)
    L = lib()
    need = ctypes.c_size_t()
    _check(L.ctcpb_lm_loss_workspace(dt, x.data_ptr(), sx, w.data_ptr(), sw, N, V, H,
                                     ctypes.byref(need)))
    on = _On(stream, dev)
    out = on.empty((2, N), torch.float32)
    ws = on.empty((need.value,), torch.uint8)
    _check(L.ctcpb_lm_loss(dt, x.data_ptr(), sx, w.data_ptr(), sw, _ptr(bias), targets.data_ptr(),
                           N, V, H, out.data_ptr(), out.data_ptr() + 4 * N, ws.data_ptr(),
                           need.value, on.ptr))
    return out[0], out[1]


def token_loss_backward(grad, x, w, targets, lse, bias=None, need=(True, True, True), stream=None):
    """Gradients (dx, dw, dbias) of sum(grad * loss) for ``token_loss_forward``
    with its lse; grad (rows,) float32.  dx and dw have x's and w's type, dbias
    is float32 (None without a bias).  `need` says which of them to compute."""
    dev, dt, N, V, H, sx, sw = _loss_args(x, w, targets, bias)
    _check_dev(grad, dev, "grad", torch.float32, (N,), contiguous=True)
    _check_dev(lse, dev, "lse", torch.float32, (N,), contiguous=True)
    L = lib()
    size = ctypes.c_size_t()
    _check(L.ctcpb_lm_loss_grad_workspace(dt, x.data_ptr(), sx, w.data_ptr(), sw, N, V, H,
                                          ctypes.byref(size)))
    on = _On(stream, dev)
    dx = on.empty((N, H), x.dtype) if need[0] else None
    dw = on.empty((V, H), w.dtype) if need[1] else None
    db = on.empty((V,), torch.float32) if need[2] and bias is not None else None
    ws = on.empty((size.value,), torch.uint8)
    _check(L.ctcpb_lm_loss_grad(dt, grad.data_ptr(), x.data_ptr(), sx, w.data_ptr(), sw,
                                _ptr(bias), targets.data_ptr(), lse.data_ptr(), N, V, H, _ptr(dx),
                                _ptr(dw), _ptr(db), ws.data_ptr(), size.value, on.ptr))
    return dx, dw, db


class _TokenLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, targets, bias):
        loss, lse = token_loss_forward(x, w, targets, bias)
        ctx.save_for_backward(x, w, targets, bias, lse)
        return loss

    @staticmethod
    def backward(ctx, grad):
        x, w, targets, bias, lse = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dw, db = token_loss_backward(grad.contiguous(), x, w, targets, lse, bias,
                                         (need[0], need[1], need[3]))
        return dx, dw, None, db


def token_loss(x, w, targets, bias=None):
    """The losses of ``token_loss_forward`` as a torch function: gradients flow
    to x, w and bias."""
    return _TokenLoss.apply(x, w, targets, bias)


class PagedCache:
    """A paged key/value cache of one attention layer and its page allocator,
    for `rows` requests of at most `max_len` tokens each.

    ``append(counts, total)`` hands out pages, ``store(k, v, slots)`` writes the
    new tokens, ``attend(q)`` attends over each request's tokens, and
    ``release(finished)`` gives pages back.  `num_pages` (default: every request
    at max_len) may be smaller: a request the pool cannot serve is flagged in
    the plan's status and holds only the tokens that have a slot.  Use one
    PagedCache per stream, or order its calls."""

    def __init__(self, rows: int, max_len: int, kv_heads: int, head_dim: int,
                 dtype=torch.bfloat16, page_size: int = 16, num_pages: int = 0, device="cuda"):
        width = -(-max_len // page_size)
        num_pages = num_pages or max(1, rows * width)
        self.page_size, self.max_len = page_size, max_len
        self.k = torch.empty((num_pages, page_size, kv_heads, head_dim), dtype=dtype, device=device)
        self.v = torch.empty_like(self.k)
        self.tables = torch.full((rows, width), -1, dtype=torch.int32, device=device)
        self.pool = torch.arange(num_pages, dtype=torch.int32, device=device)
        self.lengths = torch.zeros(rows, dtype=torch.int32, device=device)
        self.taken = torch.zeros(1, dtype=torch.int32, device=device)

    def append(self, counts, total: int, stream=None) -> CachePlan:
        plan = cache_plan(self.lengths, counts, self.tables, self.pool, self.taken,
                          self.page_size, total, stream)
        self.lengths, self.taken = plan.lengths, plan.taken
        return plan

    def store(self, k, v, slots, stream=None):
        cache_store(k, v, slots, self.k, self.v, stream)

    def attend(self, q, scale=None, window=0, max_len=0, stream=None):
        return attention(q, self.k, self.v, self.tables, self.lengths, scale, window,
                         max_len or self.max_len, stream=stream)

    def release(self, finished, stream=None):
        self.lengths, self.taken = cache_release(finished, self.lengths, self.tables, self.pool,
                                                 self.taken, self.page_size, stream)
