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
