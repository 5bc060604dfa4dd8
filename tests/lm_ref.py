"""Plain forms of the language-model operators for the tests: requests one by
one on the CPU, numbers in 64 bits."""
import math

import numpy as np
import torch


def plan(lengths, counts, tables, pool, taken, page, total):
    """cache_plan token by token.  Arguments: lists / numpy; returns a dict."""
    rows, width = tables.shape
    tables = tables.copy()
    slots, positions = [], []
    starts, after, status = [0], [], []
    for r in range(rows):
        n = min(max(int(lengths[r]), 0), width * page)
        cnt = max(int(counts[r]), 0)
        st, held = 0, n
        pages = -(-n // page)
        broken = False
        for i in range(cnt):
            at = starts[r] + i
            if at >= total:
                st |= 4
                break
            pos = n + i
            p = pos // page
            slot = -1
            if p >= width:
                st |= 2
            else:
                if p == pages:
                    pages += 1
                    if taken < len(pool):
                        tables[r, p] = pool[taken]
                    else:
                        tables[r, p] = -1
                        st |= 1
                    taken += 1
                if tables[r, p] >= 0:
                    slot = int(tables[r, p]) * page + pos % page
            if slot >= 0 and not broken:
                held = pos + 1
            else:
                broken = True
            slots.append(slot)
            positions.append(pos)
        starts.append(starts[r] + cnt)
        after.append(held)
        status.append(st)
    pad = total - len(slots)
    return dict(tables=tables, slots=np.array(slots + [-1] * pad, np.int32),
                positions=np.array(positions + [-1] * pad, np.int32),
                starts=np.array(starts, np.int32), lengths=np.array(after, np.int32),
                taken=np.array([min(taken, len(pool))], np.int32),
                status=np.array(status, np.int32))


def attention(q, k_cache, v_cache, tables, lengths, scale, window, page):
    """(out, lse, tolerance of out, tolerance of lse) in float64 on the CPU.

    The tolerances bound float32 scores and sums: a score of D products is off
    by at most (D + 4) 2^-24 of the sum of their magnitudes, so a probability by
    twice that (the maximum's error too) plus n 2^-24 for the sums and 2^-16 for
    exponentials and the two-part probabilities; the output by that times the
    largest value, plus its own rounding to `q`'s type."""
    R, Hq, D = q.shape
    Hkv = k_cache.shape[2]
    g = Hq // Hkv
    u = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}[q.dtype]
    tiny = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}[q.dtype]
    out = torch.zeros((R, Hq, D), dtype=torch.float64)
    lse = torch.full((R, Hq), -math.inf, dtype=torch.float64)
    tol_o, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    q, k_cache, v_cache = q.cpu().double(), k_cache.cpu(), v_cache.cpu()
    tables = tables.cpu()
    for r, n in enumerate(lengths.tolist()):
        n = min(max(n, 0), tables.shape[1] * page)
        lo = max(0, n - window) if window else 0
        if n == lo:
            continue
        t = torch.arange(lo, n)
        pg = tables[r].long()[t // page]
        k = k_cache[pg, t % page].double()
        v = v_cache[pg, t % page].double()
        for h in range(Hq):
            kk, vv = k[:, h // g], v[:, h // g]
            s = (kk * q[r, h]).sum(-1) * scale
            mag = float(((kk * q[r, h]).abs().sum(-1) * abs(scale)).max())
            m = s.max()
            if m == -math.inf:
                continue
            p = torch.exp(s - m)
            out[r, h] = (p[:, None] * vv).sum(0) / p.sum()
            lse[r, h] = m + torch.log(p.sum())
            e = 2 * (D + 4) * 2.0 ** -24 * mag + (n - lo + 16) * 2.0 ** -24
            tol_l[r, h] = e + 2.0 ** -22 * (1 + abs(float(lse[r, h])))
            tol_o[r, h] = (e + 2.0 ** -16) * float(vv.abs().max()) + u * out[r, h].abs() + tiny
    return out, lse, tol_o, tol_l


def loss(x, w, targets, bias, grad):
    """(loss, lse, dx, dw, dbias) in float64 on the CPU, and tolerances.

    A logit of H float32 products is off by at most e = (H + 4) 2^-24 of the sum
    of their magnitudes; loss and lse by 2e and their own rounding.  A
    probability is off by a factor 1 + 2e + 2^-17 (its exponential), d also by
    its rounding to the inputs' type (u), and the sums over n terms by n 2^-24:
    dx is off by at most |d| |w| times that, plus its own rounding; dw and dbias
    alike.  Numbers below 2^-126, the smallest normal float32 and bfloat16, may
    come out as zero."""
    u = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}[x.dtype]
    tiny = 2.0 ** -25 if x.dtype == torch.float16 else 2.0 ** -126
    X, W, t = x.cpu().double(), w.cpu().double(), targets.cpu().long()
    b = torch.zeros(W.shape[0], dtype=torch.float64) if bias is None else bias.cpu().double()
    N, H = X.shape
    V = W.shape[0]
    z = X @ W.t() + b
    e = (H + 4) * 2.0 ** -24 * (X.abs() @ W.abs().t() + b.abs()).amax(1)
    lse = torch.logsumexp(z, 1)
    ok = (t >= 0) & (t < V)
    at = torch.where(ok, t, 0)
    nll = torch.where(ok, lse - z[torch.arange(N), at], 0.0)
    tol_lse = e + 2.0 ** -21 * (1 + lse.abs())
    tol_loss = 2 * e + 2.0 ** -20 * (1 + lse.abs())
    g = torch.where(ok, grad.cpu().double(), 0.0)
    p = torch.exp(z - lse[:, None])
    hot = torch.zeros_like(p)
    hot[torch.arange(N)[ok], at[ok]] = 1
    d = g[:, None] * (p - hot)
    # the error of d: of the probability, and of rounding d to the type
    r = 2 * e + 2.0 ** -17
    de = g.abs()[:, None] * p * r[:, None] + u * d.abs()
    de += (2.0 ** -36 if x.dtype == torch.float16 else 2.0 ** -126) * g.abs().max()
    dx, dw, db = d @ W, d.t() @ X, d.sum(0)
    tol_dx = (de + V * 2.0 ** -24 * d.abs()) @ W.abs() + u * dx.abs() + tiny
    tol_dw = (de + N * 2.0 ** -24 * d.abs()).t() @ X.abs() + u * dw.abs() + tiny
    tol_db = (g.abs()[:, None] * p * r[:, None] + (N + 4) * 2.0 ** -24 * d.abs()).sum(0)
    return (nll, lse, dx, dw, db), (tol_loss, tol_lse, tol_dx, tol_dw, tol_db)
