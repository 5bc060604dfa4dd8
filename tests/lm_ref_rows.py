"""Attention of one token per request in 64 bits on the CPU, a request and
key/value head at a time, for requests too long for the plain form that goes
head by head."""
import math

import torch

ULP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def attention(q, k_cache, v_cache, tables, lengths, scale, window, page):
    """(out, lse, e, top, n) in float64: e (rows, heads) is the largest sum of the magnitudes
    of a score's products, top the largest |value| and n the tokens of each row."""
    R, Hq, D = q.shape
    Hkv = k_cache.shape[2]
    g = Hq // Hkv
    q, k_cache, v_cache, tables = q.cpu().double(), k_cache.cpu(), v_cache.cpu(), tables.cpu()
    out = torch.zeros((R, Hq, D), dtype=torch.float64)
    lse = torch.full((R, Hq), -math.inf, dtype=torch.float64)
    e, top = torch.zeros_like(lse), torch.zeros_like(lse)
    n = torch.zeros((R, 1), dtype=torch.float64)
    for r, hi in enumerate(lengths.tolist()):
        hi = min(max(hi, 0), tables.shape[1] * page)
        lo = max(0, hi - window) if window else 0
        if hi == lo:
            continue
        n[r] = hi - lo
        t = torch.arange(lo, hi)
        pg = tables[r].long()[t // page]
        k, v = k_cache[pg, t % page].double(), v_cache[pg, t % page].double()
        for h in range(Hkv):
            at = slice(h * g, (h + 1) * g)
            kk, vv = k[:, h], v[:, h]
            s = q[r, at] @ kk.t() * scale
            e[r, at] = (q[r, at].abs() @ kk.abs().t()).amax(1) * abs(scale)
            top[r, at] = vv.abs().max()
            lse[r, at] = torch.logsumexp(s, 1)
            out[r, at] = torch.softmax(s, 1) @ vv
    return out, lse, e, top, n


def tolerances(out, lse, e, top, n, D, dtype):
    """Of out and lse, for float32 scores and sums: a score of D products is off by at
    most (D + 4) 2^-24 of the sum of their magnitudes, a probability by twice that (the
    maximum's error too), n 2^-24 for the sums and 2^-16 for exponentials and the two-part
    probabilities; the output by that times the largest value, plus its own rounding."""
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
    off = 2 * (D + 4) * 2.0 ** -24 * e + (n + 16) * 2.0 ** -24
    return (((off + 2.0 ** -16) * top)[..., None] + ULP[dtype] * out.abs() + tiny,
            off + 2.0 ** -22 * (1 + lse.abs()))
