"""Plain forms of the 8-bit operators for the tests: page by page and row by row on the
CPU, numbers in 64 bits.  Codes, scales and what is read back are exact; for products the
tolerance is returned beside them."""
import math

import torch

TOP = {torch.int8: 127, torch.float8_e4m3fn: 448}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
LEAST = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}


def values(codes):
    """8-bit codes as float64 numbers, from their bits."""
    if codes.dtype == torch.int8:
        return codes.cpu().double()
    b = codes.cpu().view(torch.uint8).long()
    sign = 1.0 - 2.0 * (b >> 7).double()
    e, f = (b >> 3) & 15, (b & 7).double()
    x = torch.where(e == 0, f / 8 * 2.0 ** -6, (1 + f / 8) * torch.exp2((e - 7).double()))
    return sign * torch.where((b & 127) == 127, math.nan, x)


def nearest(y, dtype):
    """Numbers rounded to the nearest value of a code type, ties to the even one."""
    if dtype == torch.int8:
        return y.round()
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    e = torch.where(torch.exp2(e) > y.abs().clamp(min=2.0 ** -6), e - 1, e)
    step = torch.exp2(e - 3)
    return (y / step).round() * step


def unit(most, dtype):
    """The least power of two u >= 2^-126 with most <= top u; 0 for 0, NaN where not finite."""
    if not math.isfinite(most):
        return math.nan
    if most == 0:
        return 0.0
    e = -126
    while most > TOP[dtype] * 2.0 ** e:
        e += 1
    return 2.0 ** e


def store(x, slots, codes, scales):
    """(code values, scales) in float64 after x (tokens, heads, dim) went to `slots`."""
    dtype, (P, page, H, D) = codes.dtype, codes.shape
    vals, scales = values(codes), scales.cpu().double().clone()
    x, slots = x.cpu().double(), slots.cpu().tolist()
    pages = {}
    for t, s in enumerate(slots):
        if 0 <= s < P * page:
            pages.setdefault(s // page, []).append((t, s % page))
    for p, tokens in pages.items():
        for h in range(H):
            new = torch.stack([x[t, h] for t, _ in tokens])
            old = 0.0 if any(at == 0 for _, at in tokens) else float(scales[p, h])
            most = float(new.abs().max()) if not new.isnan().any() else math.nan
            need = unit(most, dtype)
            now = math.nan if math.isnan(old) or math.isnan(need) else max(old, need)
            if now > old > 0:
                vals[p, :, h] = nearest(vals[p, :, h] * (old / now), dtype)
            for (t, at), row in zip(tokens, new):
                vals[p, at, h] = nearest(row / now, dtype) if now > 0 else 0.0
            scales[p, h] = now
    return vals, scales


def load(slots, codes, scales, dtype):
    """What the slots hold, exactly rounded to `dtype`."""
    P, page, H, D = codes.shape
    every = (values(codes) * scales.cpu().double()[:, None, :, None]).flatten(0, 1)
    s = slots.cpu().long()
    there = (s >= 0) & (s < P * page)
    return torch.where(there[:, None, None], every[s.clamp(0, P * page - 1)], 0.0).to(dtype)


def quantize(x):
    """(codes, scales): exact quotients by a float32 scale, rounded in 64 bits.  (A quotient of two
    24-bit numbers that is not a half lies at least 2^-33 of itself from one: 64 bits tell.)"""
    x = x.cpu().double()
    scales = (x.abs().amax(1).float() / 127)
    bad = ~torch.isfinite(x).all(1)
    s = scales.double()[:, None]
    codes = torch.where((s > 0) & ~bad[:, None], x / s, 0.0).round().clamp(-127, 127)
    return codes, torch.where(bad, math.nan, scales)


def linear(codes, xs, w, ws, bias, dtype):
    """(result, tolerance): the sum of codes is exact and its float32 form off by 2^-24 of itself;
    two products and a sum with the bias round three times more, out once."""
    y = codes.double() @ w.cpu().double().t()
    y = y * xs.cpu().double()[:, None] * ws.cpu().double()
    b = torch.zeros(y.shape[1], dtype=torch.float64) if bias is None else bias.cpu().double()
    tol = 4 * 2.0 ** -24 * (y.abs() + b.abs()) + HALF[dtype] * (y + b).abs() + LEAST[dtype]
    return y + b, tol
