"""Cases of the second pass in 8 bits, in plain torch and through the package.

Rescoring is bound by what it reads: the key/value cache of its hypotheses and the model's
weights.  Both can be held in 8 bits.  New tokens' keys and values are quantised as they are
written, with a scale for each page and head, and read back (``store``, ``load``); one new
token per request attends over such a cache (``attention``); and a projection multiplies 8-bit
weights, scaled by channel, with activations that are quantised by token (``linear``).
"""
from __future__ import annotations

import math

import torch

own = False   # True: run() calls the package's operators instead of the plain forms

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
TOP = {"int8": 127.0, "e4m3": 448.0}   # the largest magnitude of a code


def listed():
    return [
        # one decoding step of 256 streams: a token to each one's open page, which is read back
        dict(name="store8_step", op="store", rows=256, held_hi=15, add=1, kv_heads=8, dim=128,
             dtype="bf16", code="int8", page=16, order="htd"),
        # the prompts of a batch, read back for the prompts' own attention
        dict(name="store8_prompts", op="store", rows=512, held_hi=0, add=256, kv_heads=8, dim=128,
             dtype="bf16", code="e4m3", page=16, order="thd"),
        # one document's cache back in single precision: latency
        dict(name="load8_one", op="load", tokens=500, kv_heads=8, dim=64, dtype="f32", code="int8",
             page=16, order="thd"),
        # the cache of a batch, moved to a model that keeps 16 bits
        dict(name="load8_batch", op="load", tokens=131072, kv_heads=8, dim=128, dtype="bf16",
             code="int8", page=32, order="htd"),
        # one request alone: latency
        dict(name="attn8_one", op="attention", rows=1, len_lo=500, len_hi=500, q_heads=8, kv_heads=8,
             dim=64, dtype="f32", code="int8", page=16, window=0, order="thd"),
        # a rescoring step of 128 utterances x 32 hypotheses, empty ones among them
        dict(name="attn8_nbest", op="attention", rows=4096, len_lo=0, len_hi=512, q_heads=16,
             kv_heads=4, dim=64, dtype="f16", code="e4m3", page=16, window=0, order="thd"),
        # 256 streams of very different lengths, grouped heads
        dict(name="attn8_streams", op="attention", rows=256, len_lo=1, len_hi=4096, q_heads=32,
             kv_heads=8, dim=128, dtype="bf16", code="int8", page=16, window=0, order="htd"),
        # few long documents: the length has to be split to fill the card
        dict(name="attn8_long", op="attention", rows=3, len_lo=65537, len_hi=131071, q_heads=64,
             kv_heads=8, dim=128, dtype="bf16", code="e4m3", page=64, window=0, order="htd"),
        # the output layer for one step's 32 hypotheses (latency; the weight is read once)
        dict(name="linear8_step", op="linear", rows=32, out=5000, hidden=512, dtype="bf16",
             bias=True),
        # one utterance's frames in single precision, rows of an odd length
        dict(name="linear8_odd", op="linear", rows=875, out=1531, hidden=387, dtype="f32", bias=True),
        # the last projection of a layer for all tokens of a batch of N-best lists
        dict(name="linear8_nbest", op="linear", rows=20000, out=1024, hidden=4096, dtype="f16",
             bias=False),
        # the widest projection of a larger model's layer
        dict(name="linear8_large", op="linear", rows=8192, out=8192, hidden=2048, dtype="bf16",
             bias=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("store", "load", "attention", "linear"))
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    if op == "linear":
        out, hidden = _log(rng, 29, 50000), rng.choice((_log(rng, 64, 8192), 8 * _log(rng, 8, 1024)))
        most = min(8192.0 * 8192 * 2048 / (out * hidden), 8192.0 * 8192 / out)
        rows = max(1, min(_log(rng, 1, 20000), int(most)))
        return dict(op=op, rows=rows, out=out, hidden=hidden, dtype=dtype,
                    bias=rng.choice((True, False)))
    code, order = rng.choice(("int8", "e4m3")), rng.choice(("thd", "htd"))
    kv_heads, dim = rng.choice((1, 2, 3, 4, 8)), rng.choice((64, 80, 96, 128, 256))
    page = rng.choice((4, 8, 16, 32, 64))
    most = (131072 * 8 * 128 * 2) // (kv_heads * dim * SIZE[dtype])
    if op == "store":
        rows = _log(rng, 1, 4096)
        return dict(op=op, rows=rows, held_hi=rng.choice((0, page - 1)),
                    add=rng.choice((1, _log(rng, 1, max(1, min(most, 200000) // (rows + 1))))),
                    kv_heads=kv_heads, dim=dim, dtype=dtype, code=code, page=page, order=order)
    if op == "load":
        return dict(op=op, tokens=_log(rng, 1, min(most, 200000)), kv_heads=kv_heads, dim=dim,
                    dtype=dtype, code=code, page=page, order=order)
    q_heads = kv_heads * rng.choice((1, 2, 4, 5, 8, 16))
    rows = _log(rng, 1, 4096)
    hi = _log(rng, 1, max(1, min(131072, (1 << 29) // (rows * q_heads * dim * SIZE[dtype]))))
    return dict(op=op, rows=rows, len_lo=rng.choice((0, 1, hi)), len_hi=hi, q_heads=q_heads,
                kv_heads=kv_heads, dim=dim, dtype=dtype, code=code, page=page,
                window=rng.choice((0, 0, 0, max(1, hi // 3))), order=order)


# ---------------------------------------------------------------- inputs --

def _spread(lo, hi, n):
    """n whole numbers from lo to hi, evenly spread (hi alone where n is 1)."""
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _permuted(values, seed):
    g = torch.Generator().manual_seed(seed)
    v = torch.tensor(values, dtype=torch.int64)
    return v[torch.randperm(v.numel(), generator=g)]


def _power(e):
    """2^e in 32 bits, exactly."""
    return (e.to(torch.int32) + 127 << 23).view(torch.float32)


def _cache8(pages, c, gen):
    """(codes as a (pages, page, kv_heads, dim) view, scales (pages, kv_heads)): values around
    one, kept token by token or head by head."""
    page, heads, dim = c["page"], c["kv_heads"], c["dim"]
    shape = (pages, page, heads, dim) if c["order"] == "thd" else (pages, heads, page, dim)
    x = torch.randn(shape, device="cuda", generator=gen, dtype=torch.float16)
    x *= TOP[c["code"]] / 5.0
    top = TOP[c["code"]]
    if c["code"] == "int8":
        x = x.round_()
    codes = x.clamp_(-top, top).to(CODES[c["code"]])
    if c["order"] == "htd":
        codes = codes.transpose(1, 2)
    e = torch.randint(-2, 2, (pages, heads), device="cuda", generator=gen)
    unit = -5 if c["code"] == "int8" else -7
    return codes, _power(e + unit)


def _starts(per_row):
    return per_row.cumsum(0) - per_row


def _ranges(first, count):
    """first[r], first[r] + 1, ... for count[r] numbers of every row r, one after another."""
    row = torch.repeat_interleave(torch.arange(count.numel()), count)
    return row, first[row] + torch.arange(row.numel()) - _starts(count)[row]


def prepare(case, seed):
    c, dev = dict(case), "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    s = {"case": c}
    dtype = DTYPES[c["dtype"]]
    g = torch.Generator().manual_seed(seed + 7)
    if c["op"] == "linear":
        N, V, H = c["rows"], c["out"], c["hidden"]
        size = torch.exp(0.5 * torch.randn((N, 1), device=dev, generator=gen))   # loud and quiet tokens
        s["x"] = (torch.randn((N, H), device=dev, generator=gen) * size).to(dtype)
        w = torch.randn((V, H), device=dev, generator=gen) * (3 / math.sqrt(H))
        s["w_scale"] = w.abs().amax(1) / 127.0
        # 8-bit weights with rows on 16 bytes, as a user keeps them
        s["w"] = torch.zeros((V, -(-H // 16) * 16), dtype=torch.int8, device=dev)[:, :H]
        s["w"].copy_((w / s["w_scale"][:, None]).round_().clamp_(-127, 127))
        s["bias"] = torch.randn((V,), device=dev, generator=gen) if c["bias"] else None
        return s
    page = c["page"]
    if c["op"] == "store":
        # row r's open page holds held[r] tokens, and `add` more come
        held = _permuted(_spread(0, min(c["held_hi"], page - 1), c["rows"]), seed)
        touched = (held + c["add"] + page - 1) // page
        pages = int(touched.sum()) + 3
        ids = torch.randperm(pages, generator=g)
        row, pos = _ranges(held, torch.full_like(held, c["add"]))
        slots = ids[_starts(touched)[row] + pos // page] * page + pos % page
        slots[torch.rand(slots.numel(), generator=g) < 0.02] = -1   # a few tokens without a slot
        row, pos = _ranges(torch.zeros_like(held), held)
        before = ids[_starts(touched)[row]] * page + pos
        s["slots"] = slots.to(dev, torch.int32)
        s["read"] = torch.cat((before, slots)).to(dev, torch.int32)
        s["k_cache"], s["k_scale"] = _cache8(pages, c, gen)
        s["v_cache"], s["v_scale"] = _cache8(pages, c, gen)
        # keys and values as a fused projection leaves them: two slices of one tensor
        s["kv"] = torch.randn((slots.numel(), 2, c["kv_heads"], c["dim"]), device=dev, generator=gen,
                              dtype=dtype)
        return s
    if c["op"] == "load":
        T = c["tokens"]
        pages = -(-T // page) + 3
        s["k_cache"], s["k_scale"] = _cache8(pages, c, gen)
        s["v_cache"], s["v_scale"] = _cache8(pages, c, gen)
        slots = torch.arange(pages * page, dtype=torch.int32).view(pages, page)
        slots = slots[torch.randperm(pages, generator=g)].reshape(-1)[:T].clone()
        slots[torch.rand(T, generator=g) < 0.02] = -1
        s["slots"] = slots.to(dev)
        return s
    R = c["rows"]
    lens = _permuted(_spread(c["len_lo"], c["len_hi"], R), seed)
    have = (lens + page - 1) // page
    width, pages = -(-c["len_hi"] // page), int(have.sum()) + 2
    ids = torch.randperm(pages, generator=g)
    tables = torch.full((R, width), -1, dtype=torch.int64)
    row, k = _ranges(torch.zeros_like(have), have)
    tables[row, k] = ids[:row.numel()]
    s["lengths"], s["tables"] = lens.to(dev, torch.int32), tables.to(dev, torch.int32)
    s["k_cache"], s["k_scale"] = _cache8(pages, c, gen)
    s["v_cache"], s["v_scale"] = _cache8(pages, c, gen)
    s["q"] = 2 * torch.randn((R, c["q_heads"], c["dim"]), device=dev, generator=gen, dtype=dtype)
    s["scale"] = c["dim"] ** -0.5
    return s


# ----------------------------------------------------------- plain forms --

def _bytes(cache):
    return cache.view(torch.uint8)   # indexing works for it on every tree


def _values(cache, scale, pg, at):
    """Values of cache[pg, at] in 32 bits."""
    codes = _bytes(cache)[pg, at].view(cache.dtype)
    return codes.float() * scale[pg][..., None]


def _store_one(x, slots, cache, scale, top):
    """Quantises x (tokens, heads, dim) into a cache and its scales, both changed in place."""
    P, page = cache.shape[:2]
    keep = slots >= 0
    x, slots = x[keep].float(), slots[keep].long()
    pg, at = slots // page, slots % page
    most = torch.zeros_like(scale).scatter_reduce(
        0, pg[:, None].expand(-1, scale.shape[1]), x.abs().amax(-1), "amax")
    # the least power of two whose multiple by the largest code holds the largest value
    mant, e = torch.frexp(most.double() / top)
    e = torch.where(mant == 0.5, e - 1, e).clamp(min=-126)
    need = torch.where(most > 0, _power(e), 0.0)
    begun = torch.zeros(P, dtype=torch.bool, device=x.device)
    begun[pg[at == 0]] = True
    old = torch.where(begun[:, None], 0.0, scale)
    new = torch.maximum(old, need)
    grown = torch.nonzero(((new > old) & (old > 0)).any(1))[:, 0]   # what is there is rescaled
    ratio = torch.where(new > 0, old / new, 1.0)[grown][:, None, :, None]
    codes = _bytes(cache)[grown].view(cache.dtype).float() * ratio
    whole = cache.dtype == torch.int8
    _bytes(cache)[grown] = _bytes((codes.round() if whole else codes).to(cache.dtype))
    unit = new[pg][..., None]
    codes = torch.where(unit > 0, x / unit, 0.0)
    _bytes(cache)[pg, at] = _bytes((codes.round() if whole else codes).to(cache.dtype))
    touched = torch.zeros(P, dtype=torch.bool, device=x.device)
    touched[pg] = True
    scale.copy_(torch.where(touched[:, None], new, scale))


def _store(s):
    top = TOP[s["case"]["code"]]
    _store_one(s["kv"][:, 0], s["slots"], s["k_cache"], s["k_scale"], top)
    _store_one(s["kv"][:, 1], s["slots"], s["v_cache"], s["v_scale"], top)
    got = _load(s, s["read"])
    got["k_scale"], got["v_scale"] = s["k_scale"], s["v_scale"]
    return got


def _load(s, slots):
    page, dtype = s["case"]["page"], DTYPES[s["case"]["dtype"]]
    there = (slots >= 0)[:, None, None]
    slots = slots.long().clamp(min=0)
    got = {}
    for name in ("k", "v"):
        x = _values(s[name + "_cache"], s[name + "_scale"], slots // page, slots % page)
        got[name] = torch.where(there, x, 0.0).to(dtype)
    return got


def _attention(s):
    c = s["case"]
    page, lens, q = c["page"], s["lengths"].long(), s["q"].float()
    R, Hq, D = q.shape
    Hkv, L = c["kv_heads"], c["len_hi"]
    t = torch.arange(L, device=q.device)
    keep = t < lens[:, None]
    if c["window"]:
        keep &= t >= lens[:, None] - c["window"]
    pg = s["tables"].long()[:, t // page].clamp(min=0)
    k = _values(s["k_cache"], s["k_scale"], pg, t % page).permute(0, 2, 3, 1).contiguous()
    scores = torch.matmul(q.view(R, Hkv, Hq // Hkv, D), k) * s["scale"]
    del k
    scores = torch.where(keep[:, None, None, :], scores, -math.inf)
    m = scores.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(scores - m)
    del scores
    total = p.sum(-1, keepdim=True)
    v = _values(s["v_cache"], s["v_scale"], pg, t % page)
    v = torch.where(keep[:, :, None, None], v, 0.0)
    out = torch.matmul(p, v.permute(0, 2, 1, 3).contiguous())
    out = torch.where(total == 0, 0.0, out / total)
    lse = (m + torch.log(total)).view(R, Hq)
    return {"out": out.view(R, Hq, D).to(s["q"].dtype), "lse": lse}


def _linear(s):
    x = s["x"].float()
    unit = x.abs().amax(1, keepdim=True) / 127.0
    # quotients next to a half have to fall on their own side
    codes = torch.where(unit > 0, x.double() / unit.double(), 0.0).round().clamp(-127, 127).float()
    y = torch.matmul(codes, s["w"].float().t())
    y = y * unit * s["w_scale"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return {"out": y.to(s["x"].dtype)}


def _run_own(s):
    from ctc_prefix_beam_amd import lm
    c = s["case"]
    if c["op"] == "linear":
        return {"out": lm.linear8(s["x"], s["w"], s["w_scale"], s["bias"])}
    cache = (s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    if c["op"] == "attention":
        out, lse = lm.attention8(s["q"], *cache, s["tables"], s["lengths"], scale=s["scale"],
                                 window=c["window"])
        return {"out": out, "lse": lse}
    if c["op"] == "load":
        k, v = lm.cache_load8(s["slots"], *cache, dtype=DTYPES[c["dtype"]])
        return {"k": k, "v": v}
    lm.cache_store8(s["kv"][:, 0], s["kv"][:, 1], s["slots"], *cache)
    k, v = lm.cache_load8(s["read"], *cache, dtype=DTYPES[c["dtype"]])
    return {"k": k, "v": v, "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "store":
        return _store(state)
    if op == "load":
        return _load(state, state["slots"])
    if op == "attention":
        return _attention(state)
    return _linear(state)


def work(case):
    c = case
    if c["op"] == "linear":
        N, V, H = float(c["rows"]), float(c["out"]), float(c["hidden"])
        return {"bytes": N * H * SIZE[c["dtype"]] + V * H + N * V * SIZE[c["dtype"]] + 4 * V,
                "flops": 2 * N * V * H}
    row = 2.0 * c["kv_heads"] * c["dim"]   # values of a token's keys and values
    one = SIZE[c["dtype"]]
    if c["op"] == "load":
        return {"bytes": c["tokens"] * (row * (1 + one) + 4), "flops": 0}
    if c["op"] == "store":
        held = sum(_spread(0, min(c["held_hi"], c["page"] - 1), c["rows"]))
        new = float(c["rows"] * c["add"])
        # written once from the inputs, and read back with what was there
        return {"bytes": new * (row * (one + 1) + 4) + (new + held) * (row * (1 + one) + 4),
                "flops": 0}
    lens = _spread(c["len_lo"], c["len_hi"], c["rows"])
    seen = float(sum(min(n, c["window"]) if c["window"] else n for n in lens))
    q = 2.0 * c["rows"] * c["q_heads"] * c["dim"] * one
    return {"bytes": seen * row * (1 + 4.0 / (c["page"] * c["dim"])) + q,
            "flops": 4 * seen * c["q_heads"] * c["dim"]}


# ---------------------------------------------------------------- exact --

def _exact_codes(y, code):
    """Numbers rounded to the nearest code, ties to the even one."""
    if code == "int8":
        return y.round()
    e = torch.frexp(y)[1].clamp(min=-5) - 1          # 2^e <= |y|, or the smallest normal
    step = (e.long() + 1020 << 52).view(torch.float64)   # 2^(e - 3)
    return (y / step).round() * step


def _exact_unit(most, top):
    """The least power of two with most <= top * it (0 for 0)."""
    e = torch.log2(most / top).ceil().clamp(-126, 128)
    unit = (e.long() + 1023 << 52).view(torch.float64)
    unit = torch.where((e > -126) & (most <= top * unit / 2), unit / 2, unit)
    unit = torch.where(most > top * unit, unit * 2, unit)
    return torch.where(most == 0, 0.0, unit)


def _exact_store(s, x, cache, scale):
    c = s["case"]
    P, page, H, D = cache.shape
    slots = s["slots"].long()
    # a last page for the tokens without a slot
    at = torch.where(slots >= 0, slots, P * page)
    new = torch.zeros(((P + 1) * page, H, D), dtype=torch.float64, device="cuda")
    new[at] = x.double()
    there = torch.zeros((P + 1) * page, dtype=torch.bool, device="cuda")
    there[at] = True
    new, there = new[:P * page].view(P, page, H, D), there[:P * page].view(P, page)
    old = torch.where(there[:, :1], 0.0, scale.double())
    unit = torch.maximum(old, _exact_unit(new.abs().amax((1, 3)), TOP[c["code"]]))
    unit = torch.where(there.any(1)[:, None], unit, scale.double())
    was = cache.double() * torch.where(unit > 0, old / unit, 0.0)[:, None, :, None]
    got = torch.where(there[..., None, None], new / unit[:, None, :, None], was)
    got = torch.where(unit[:, None, :, None] > 0, got, 0.0)
    return (_exact_codes(got, c["code"]) * unit[:, None, :, None]).flatten(0, 1), unit


def exact(case, seed):
    """The computed outputs from the definition in 64 bits."""
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "linear":
        got = torch.empty((c["rows"], c["out"]), dtype=torch.float64, device="cuda")
        w = s["w"].double() * s["w_scale"].double()[:, None]
        for a in range(0, c["rows"], 2048):
            x = s["x"][a:a + 2048].double()
            # a scale is a float32 number
            unit = (x.abs().amax(1) / 127).float().double()
            n = (x / torch.where(unit > 0, unit, 1.0)[:, None]).clamp(-127, 127).round()
            got[a:a + 2048] = torch.mm(n * unit[:, None], w.t())
        if s["bias"] is not None:
            got += s["bias"].double()
        return {"out": got}
    if c["op"] == "store":
        slots = s["read"].long()
        got = {}
        for i, name in enumerate(("k", "v")):
            x, unit = _exact_store(s, s["kv"][:, i], s[name + "_cache"], s[name + "_scale"])
            got[name] = torch.where((slots >= 0)[:, None, None], x[slots.clamp(min=0)], 0.0)
            got[name + "_scale"] = unit
        return {n: got[n] for n in ("k", "v", "k_scale", "v_scale")}
    if c["op"] == "load":
        slots = s["slots"].long()
        got = {}
        for name in ("k", "v"):
            x = s[name + "_cache"].double() * s[name + "_scale"].double()[:, None, :, None]
            x = x.flatten(0, 1)[slots.clamp(min=0)]
            got[name] = torch.where((slots >= 0)[:, None, None], x, 0.0)
        return got
    page, g = c["page"], c["q_heads"] // c["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for r, n in enumerate(s["lengths"].tolist()):
        if n == 0:
            continue
        lo = max(0, n - c["window"]) if c["window"] else 0
        pg = s["tables"][r, lo // page:(n - 1) // page + 1].long()
        first = lo - lo // page * page
        k, v = (_bytes(s[name + "_cache"])[pg].view(s[name + "_cache"].dtype).double() *
                s[name + "_scale"][pg].double()[:, None, :, None] for name in ("k", "v"))
        k = k.flatten(0, 1)[first:first + n - lo]    # n, Hkv, D
        v = v.flatten(0, 1)[first:first + n - lo]
        for h in range(c["kv_heads"]):
            z = torch.mm(s["q"][r, h * g:(h + 1) * g].double(), k[:, h].t().contiguous())
            z *= s["scale"]
            lse[r, h * g:(h + 1) * g] = torch.logsumexp(z, -1)
            out[r, h * g:(h + 1) * g] = torch.mm(torch.softmax(z, -1), v[:, h].contiguous())
    return {"out": out, "lse": lse}
