"""Operators for rescoring N-best lists with a language model on MI355X.

Thin Python binding of ``libctcpb_lm.so`` (C ABI in ``include/ctcpb_lm.h``):
the pages and slots of a paged key/value cache from device-resident lengths
(``cache_plan``, ``cache_release``), the store of new tokens' keys and values
(``cache_store``), the attention of one new token per request over the cache
(``attention``), and token losses over a large vocabulary without keeping the
logits, with their gradients (``token_loss``).  ``PagedCache`` holds the tensors
of a cache.  Every step runs in the library's HIP kernels; PyTorch provides
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
           "ctcpb_lm_last_error")
NO_PAGE, NO_ENTRY, NO_SLOT = 1, 2, 4   # status bits of cache_plan
_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_SPLIT_D = 256   # CTCPB_LM_SPLIT_D

# The argument structures of include/ctcpb_lm.h, in order (native sizes and
# alignment): a call packs them once instead of converting each argument.
_PLAN = struct.Struct("11Pq5i4x")
_RELEASE = struct.Struct("7Pq4i")
_STORE = struct.Struct("3P4qP3qP3q6i")
_ATTENTION = struct.Struct("5P5qP3qP3q10if4x")
_LOSS = struct.Struct("6P2q4i")
_GRAD = struct.Struct("9P2q4i")

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
        for name in ("cache_plan", "cache_release", "cache_store"):
            getattr(L, "ctcpb_lm_" + name).argtypes = [args, p]
        for name in ("attention", "loss", "loss_grad"):
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
        width = -(-max_len // page_size)
        num_pages = num_pages or max(1, rows * width)
        self.page_size, self.max_len = page_size, width * page_size
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

    def store(self, k, v, slots, layer: int = 0, stream=None):
        cache_store(k, v, slots, self.k[layer], self.v[layer], stream)
        self._keep(stream, self.k, self.v)

    def attend(self, q, layer: int = 0, scale=None, window: int = 0, max_len: int = 0, stream=None):
        got = attention(q, self.k[layer], self.v[layer], self.tables, self.lengths, scale, window,
                        max_len, stream=stream)
        self._keep(stream, self.k, self.v, self.tables, self.lengths)
        return got

    def release(self, finished, stream=None):
        lengths, taken = cache_release(finished, self.lengths, self.tables, self.pool, self.taken,
                                       self.page_size, stream)
        self._keep(stream, self.lengths, self.taken, self.tables, self.pool)
        self.lengths, self.taken = lengths, taken
