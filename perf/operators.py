"""Cases of the operators behind N-best rescoring, in plain torch and through the package.

The decoder's hypotheses are rescored by a language model token by token: the pages of its
key/value cache are handed out from the request lengths (``plan``), the new tokens' keys and
values go to their slots (``store``), one new token per request attends over the paged cache
(``attention``), and the output layer gives each token's loss over the vocabulary without
keeping the logits (``loss``), with the gradients when that layer is trained (``grad``).
"""
from __future__ import annotations

import math

import torch

own = False   # True: run() calls the package's operators instead of the plain forms

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # one decoding step of 256 streams: every stream appends one token
        dict(name="plan_step", op="plan", rows=256, len_lo=0, len_hi=4095, cnt_lo=1, cnt_hi=1,
             page=16, short=0),
        # the prompts of 128 utterances x 32 hypotheses at once, some of them empty
        dict(name="plan_prompts", op="plan", rows=4096, len_lo=0, len_hi=0, cnt_lo=0, cnt_hi=512,
             page=16, short=0),
        # the keys and values of that decoding step's 256 tokens
        dict(name="store_step", op="store", tokens=256, kv_heads=8, dim=128, dtype="bf16", page=16,
             order="thd"),
        # the keys and values of a batch of prompts, a few tokens without a slot
        dict(name="store_prompts", op="store", tokens=131072, kv_heads=8, dim=128, dtype="bf16",
             page=16, order="thd"),
        # one request alone: latency
        dict(name="attn_one", op="attention", rows=1, len_lo=500, len_hi=500, q_heads=8, kv_heads=8,
             dim=64, dtype="f32", page=16, window=0, order="thd"),
        # a rescoring step of 128 utterances x 32 hypotheses, empty ones among them
        dict(name="attn_nbest", op="attention", rows=4096, len_lo=0, len_hi=512, q_heads=16,
             kv_heads=4, dim=64, dtype="f16", page=16, window=0, order="thd"),
        # 256 streams of very different lengths, grouped heads
        dict(name="attn_streams", op="attention", rows=256, len_lo=1, len_hi=4096, q_heads=32,
             kv_heads=8, dim=128, dtype="bf16", page=16, window=0, order="thd"),
        # few long documents: the length has to be split to fill the card
        dict(name="attn_long", op="attention", rows=3, len_lo=65537, len_hi=131071, q_heads=64,
             kv_heads=8, dim=128, dtype="bf16", page=64, window=0, order="htd"),
        # the scores of one step's 32 hypotheses (latency; the weight is read once)
        dict(name="loss_step", op="loss", rows=32, vocab=5000, hidden=512, dtype="bf16", bias=True),
        # the scores of all tokens of a batch of N-best lists
        dict(name="loss_nbest", op="loss", rows=20000, vocab=5000, hidden=1024, dtype="bf16",
             bias=True),
        # a training step of the output layer over a large vocabulary
        dict(name="grad_large", op="grad", rows=8192, vocab=50000, hidden=2048, dtype="bf16",
             bias=False),
        # the same in single precision at one utterance's frames
        dict(name="grad_f32", op="grad", rows=875, vocab=5000, hidden=384, dtype="f32", bias=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("plan", "store", "attention", "loss", "grad"))
    if op == "plan":
        rows = _log(rng, 1, 4096)
        most = max(1, min(4096, (1 << 20) // rows))
        cnt = _log(rng, 1, most)
        return dict(op=op, rows=rows, len_lo=0, len_hi=_log(rng, 1, 4096), cnt_lo=rng.choice((0, cnt)),
                    cnt_hi=cnt, page=rng.choice((4, 8, 16, 32, 64)), short=rng.choice((0, 0, 1)))
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    order = rng.choice(("thd", "htd"))
    kv_heads, dim = rng.choice((1, 2, 3, 4, 8)), rng.choice((64, 80, 96, 128, 256))
    if op == "store":
        most = (131072 * 8 * 128 * 2) // (kv_heads * dim * SIZE[dtype])
        return dict(op=op, tokens=_log(rng, 1, min(most, 200000)), kv_heads=kv_heads, dim=dim,
                    dtype=dtype, page=rng.choice((4, 8, 16, 32, 64)), order=order)
    if op == "attention":
        q_heads = kv_heads * rng.choice((1, 2, 4, 5, 8, 16))
        rows = _log(rng, 1, 4096)
        most = (1 << 29) // (rows * q_heads * dim * SIZE[dtype])
        hi = _log(rng, 1, max(1, min(131072, most)))
        return dict(op=op, rows=rows, len_lo=rng.choice((0, 1, hi)), len_hi=hi, q_heads=q_heads,
                    kv_heads=kv_heads, dim=dim, dtype=dtype, page=rng.choice((4, 8, 16, 32, 64)),
                    window=rng.choice((0, 0, 0, max(1, hi // 3))), order=order)
    rows, vocab = _log(rng, 1, 20000), _log(rng, 29, 50000)
    hidden = rng.choice((_log(rng, 64, 2048), 8 * _log(rng, 8, 256)))
    most = {"loss": 1e11, "grad": 8192.0 * 50000 * 2048}[op] / (8 if dtype == "f32" else 1)
    rows = max(1, min(rows, int(most / (vocab * hidden))))
    return dict(op=op, rows=rows, vocab=vocab, hidden=hidden, dtype=dtype,
                bias=rng.choice((True, False)))


# ---------------------------------------------------------------- inputs --

def _spread(lo, hi, n):
    """n whole numbers from lo to hi, evenly spread (hi alone where n is 1)."""
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _permuted(values, seed):
    g = torch.Generator().manual_seed(seed)
    v = torch.tensor(values, dtype=torch.int32)
    return v[torch.randperm(v.numel(), generator=g)]


def _held_pages(lengths, page, width, pages, seed):
    """(tables, pool): the pages of `lengths` tokens per row at the front of a shuffled pool."""
    dev = lengths.device
    g = torch.Generator().manual_seed(seed + 7)
    pool = torch.randperm(pages, generator=g).to(torch.int32).to(dev)
    have = (lengths.long() + page - 1) // page
    off = have.cumsum(0) - have
    k = torch.arange(width, device=dev)
    at = (off[:, None] + k).clamp(max=max(pages - 1, 0))
    tables = torch.where(k < have[:, None], pool[at], torch.full((), -1, dtype=torch.int32, device=dev))
    return tables.contiguous(), pool, int(have.sum())


def _cache(pages, page, kv_heads, dim, dtype, order, gen):
    """(pages, page, kv_heads, dim) view of a cache kept token by token or head by head."""
    if order == "thd":
        return torch.randn((pages, page, kv_heads, dim), device="cuda", generator=gen, dtype=dtype)
    return torch.randn((pages, kv_heads, page, dim), device="cuda", generator=gen,
                       dtype=dtype).transpose(1, 2)


def prepare(case, seed):
    c, dev = dict(case), "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    s = {"case": c}
    if c["op"] == "plan":
        R, page = c["rows"], c["page"]
        lens = _permuted(_spread(c["len_lo"], c["len_hi"], R), seed)
        cnts = _permuted(_spread(c["cnt_lo"], c["cnt_hi"], R), seed + 1)
        width = -(-(c["len_hi"] + c["cnt_hi"]) // page)
        total = int((-(-(lens.long() + cnts.long()) // page)).sum())
        held = int((-(-lens.long() // page)).sum())
        # `short`: a pool with too few pages for the last rows
        pages = held + (total - held) // 2 if c["short"] else total + 8
        s["lengths"], s["counts"] = lens.to(dev), cnts.to(dev)
        s["tables"], s["pool"], taken = _held_pages(s["lengths"], page, width, max(pages, 1), seed)
        s["taken"] = torch.tensor([taken], dtype=torch.int32, device=dev)
        s["total"] = int(cnts.sum())
        return s
    dtype = DTYPES.get(c["dtype"])
    if c["op"] == "store":
        T, page = c["tokens"], c["page"]
        pages = -(-T // page) + 3
        s["k_cache"] = _cache(pages, page, c["kv_heads"], c["dim"], dtype, c["order"], gen)
        s["v_cache"] = _cache(pages, page, c["kv_heads"], c["dim"], dtype, c["order"], gen)
        # keys and values as a fused projection leaves them: two slices of one tensor
        s["kv"] = torch.randn((T, 2, c["kv_heads"], c["dim"]), device=dev, generator=gen, dtype=dtype)
        g = torch.Generator().manual_seed(seed)
        slots = torch.arange(pages * page, dtype=torch.int32).view(pages, page)
        slots = slots[torch.randperm(pages, generator=g)].reshape(-1)[:T].clone()
        slots[torch.rand(T, generator=g) < 0.02] = -1
        s["slots"] = slots.to(dev)
        return s
    if c["op"] == "attention":
        R, page = c["rows"], c["page"]
        lens = _permuted(_spread(c["len_lo"], c["len_hi"], R), seed)
        width = -(-c["len_hi"] // page)
        pages = int((-(-lens.long() // page)).sum()) + 2
        s["lengths"] = lens.to(dev)
        s["tables"], _, _ = _held_pages(s["lengths"], page, width, pages, seed)
        s["k_cache"] = _cache(pages, page, c["kv_heads"], c["dim"], dtype, c["order"], gen)
        s["v_cache"] = _cache(pages, page, c["kv_heads"], c["dim"], dtype, c["order"], gen)
        s["q"] = 2 * torch.randn((R, c["q_heads"], c["dim"]), device=dev, generator=gen, dtype=dtype)
        s["scale"] = c["dim"] ** -0.5
        return s
    N, V, H = c["rows"], c["vocab"], c["hidden"]
    s["x"] = torch.randn((N, H), device=dev, generator=gen, dtype=dtype)
    s["w"] = (torch.randn((V, H), device=dev, generator=gen) * (3 / math.sqrt(H))).to(dtype)
    s["bias"] = torch.randn((V,), device=dev, generator=gen) if c["bias"] else None
    t = torch.randint(0, V, (N,), device=dev, generator=gen, dtype=torch.int32)
    # one in ten is the decoder's -1 padding
    s["targets"] = torch.where(torch.rand((N,), device=dev, generator=gen) < 0.1, -1, t).to(torch.int32)
    # weights of the rows' losses, of either sign (a risk over the N best), with a loss
    # scale for half precision
    g = torch.rand((N,), device=dev, generator=gen) * 2 - 1
    s["grad"] = g * ((1024.0 if c["dtype"] == "f16" else 1.0) / N)
    return s


# ----------------------------------------------------------- plain forms --

def _plan(s):
    c = s["case"]
    page, lens, cnts, tables = c["page"], s["lengths"].long(), s["counts"].long(), s["tables"]
    R, P = tables.shape
    F, S, dev = s["pool"].numel(), s["total"], lens.device
    have = (lens + page - 1) // page
    need = ((lens + cnts + page - 1) // page).clamp(max=P) - have
    off = need.cumsum(0) - need
    taken = s["taken"].long()
    k = torch.arange(P, device=dev)
    at = taken + off[:, None] + k - have[:, None]
    fresh = torch.where(at < F, s["pool"][at.clamp(0, F - 1)], -1)
    isnew = (k >= have[:, None]) & (k < (have + need)[:, None])
    out = torch.where(isnew, fresh, tables).to(torch.int32)
    got = torch.minimum(need, (F - taken - off).clamp(min=0))
    lengths = torch.minimum(lens + cnts, (have + got) * page)
    starts = torch.zeros(R + 1, dtype=torch.int64, device=dev)
    starts[1:] = cnts.cumsum(0)
    j = torch.arange(S, device=dev)
    r = torch.searchsorted(starts[1:].contiguous(), j, right=True)
    pos = lens[r] + j - starts[r]
    pg = out[r, (pos // page).clamp(max=P - 1)].long()
    slots = torch.where((pg >= 0) & (pos < P * page), pg * page + pos % page, -1)
    status = (got < need).int() + 2 * (lens + cnts > P * page).int()
    return {"tables": out, "slots": slots.int(), "positions": pos.int(), "starts": starts.int(),
            "lengths": lengths.int(), "taken": (taken + need.sum()).clamp(max=F).int(),
            "status": status.int()}


def _store(s):
    slots = s["slots"].long()
    keep = slots >= 0
    page = s["case"]["page"]
    at = slots[keep]
    s["k_cache"][at // page, at % page] = s["kv"][:, 0][keep]
    s["v_cache"][at // page, at % page] = s["kv"][:, 1][keep]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


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
    k = s["k_cache"][pg, t % page].float().permute(0, 2, 3, 1).contiguous()      # R, Hkv, D, L
    scores = torch.matmul(q.view(R, Hkv, Hq // Hkv, D), k) * s["scale"]
    del k
    scores = torch.where(keep[:, None, None, :], scores, -math.inf)
    m = scores.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(scores - m)
    total = p.sum(-1, keepdim=True)
    v = torch.where(keep[:, :, None, None], s["v_cache"][pg, t % page].float(), 0.0)
    out = torch.matmul(p, v.permute(0, 2, 1, 3).contiguous())
    out = torch.where(total == 0, 0.0, out / total)
    lse = (m + torch.log(total)).view(R, Hq)
    return {"out": out.view(R, Hq, D).to(s["q"].dtype), "lse": lse}


def _loss(s, grads):
    x, w, t = s["x"].float(), s["w"].float(), s["targets"].long()
    V = w.shape[0]
    valid = (t >= 0) & (t < V)
    at = torch.where(valid, t, 0)[:, None]
    logits = torch.matmul(x, w.t())
    if s["bias"] is not None:
        logits += s["bias"]
    m = logits.amax(-1, keepdim=True)
    lse = m + torch.log(torch.exp(logits - m).sum(-1, keepdim=True))
    loss = torch.where(valid, (lse - logits.gather(1, at))[:, 0], 0.0)
    if not grads:
        return {"loss": loss, "lse": lse[:, 0]}
    g = torch.where(valid, s["grad"], 0.0)[:, None]
    d = torch.exp(logits - lse)
    del logits
    d.scatter_add_(1, at, torch.full_like(g, -1.0))
    d *= g
    got = {"loss": loss, "dx": torch.matmul(d, w).to(s["x"].dtype),
           "dw": torch.matmul(d.t(), x).to(s["w"].dtype)}
    if s["bias"] is not None:
        got["dbias"] = d.sum(0)
    return got


def _run_own(s):
    from ctc_prefix_beam_amd import lm
    c = s["case"]
    if c["op"] == "plan":
        p = lm.cache_plan(s["lengths"], s["counts"], s["tables"], s["pool"], s["taken"], c["page"],
                          s["total"])
        return {"tables": s["tables"], "slots": p.slots, "positions": p.positions,
                "starts": p.starts, "lengths": p.lengths, "taken": p.taken, "status": p.status}
    if c["op"] == "store":
        lm.cache_store(s["kv"][:, 0], s["kv"][:, 1], s["slots"], s["k_cache"], s["v_cache"])
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if c["op"] == "attention":
        out, lse = lm.attention(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lengths"],
                                scale=s["scale"], window=c["window"])
        return {"out": out, "lse": lse}
    loss, lse = lm.token_loss_forward(s["x"], s["w"], s["targets"], s["bias"])
    if c["op"] == "loss":
        return {"loss": loss, "lse": lse}
    dx, dw, db = lm.token_loss_backward(s["grad"], s["x"], s["w"], s["targets"], lse, s["bias"])
    got = {"loss": loss, "dx": dx, "dw": dw}
    if s["bias"] is not None:
        got["dbias"] = db
    return got


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "plan":
        return _plan(state)
    if op == "store":
        return _store(state)
    if op == "attention":
        return _attention(state)
    return _loss(state, op == "grad")


def work(case):
    c = case
    if c["op"] == "plan":
        R, page = c["rows"], c["page"]
        tokens = sum(_spread(c["cnt_lo"], c["cnt_hi"], R))
        # lengths, counts, their updates, starts and status; slots and positions; each page's
        # entry read from the pool and written to its table
        return {"bytes": 24.0 * R + 8.0 * tokens + 8.0 * max(1, tokens // page), "flops": 0}
    if c["op"] == "store":
        return {"bytes": 4.0 * c["tokens"] * c["kv_heads"] * c["dim"] * SIZE[c["dtype"]], "flops": 0}
    if c["op"] == "attention":
        lens = _spread(c["len_lo"], c["len_hi"], c["rows"])
        seen = float(sum(min(n, c["window"]) if c["window"] else n for n in lens))
        q = 2.0 * c["rows"] * c["q_heads"] * c["dim"] * SIZE[c["dtype"]]
        return {"bytes": 2 * seen * c["kv_heads"] * c["dim"] * SIZE[c["dtype"]] + q,
                "flops": 4 * seen * c["q_heads"] * c["dim"]}
    N, V, H = float(c["rows"]), float(c["vocab"]), float(c["hidden"])
    move = (N + V) * H * SIZE[c["dtype"]]
    if c["op"] == "loss":
        return {"bytes": move + 12 * N, "flops": 2 * N * V * H}
    return {"bytes": 2 * move + 12 * N, "flops": 6 * N * V * H}   # each of the three products once


# ---------------------------------------------------------------- exact --

def exact(case, seed):
    """The computed outputs from the definition in 64 bits (row by row or in blocks of rows)."""
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] in ("plan", "store"):
        return None
    if c["op"] == "attention":
        page, g = c["page"], c["q_heads"] // c["kv_heads"]
        lens = s["lengths"].tolist()
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
        for r, n in enumerate(lens):
            if n == 0:
                continue
            lo = max(0, n - c["window"]) if c["window"] else 0
            pg = s["tables"][r, lo // page:(n - 1) // page + 1].long()
            first = lo - lo // page * page
            k = s["k_cache"][pg].flatten(0, 1)[first:first + n - lo].double()    # n, Hkv, D
            v = s["v_cache"][pg].flatten(0, 1)[first:first + n - lo].double()
            for h in range(c["kv_heads"]):
                z = torch.mm(s["q"][r, h * g:(h + 1) * g].double(), k[:, h].t().contiguous())
                z *= s["scale"]
                lse[r, h * g:(h + 1) * g] = torch.logsumexp(z, -1)
                out[r, h * g:(h + 1) * g] = torch.mm(torch.softmax(z, -1), v[:, h].contiguous())
        return {"out": out, "lse": lse}
    N, V, H = c["rows"], c["vocab"], c["hidden"]
    if (2 if c["op"] == "loss" else 6) * float(N) * V * H > 1e14:
        return None
    w = s["w"].double()
    loss = torch.zeros(N, dtype=torch.float64, device="cuda")
    lses = torch.zeros(N, dtype=torch.float64, device="cuda")
    dx = torch.zeros((N, H), dtype=torch.float64, device="cuda")
    dw = torch.zeros((V, H), dtype=torch.float64, device="cuda")
    db = torch.zeros(V, dtype=torch.float64, device="cuda")
    for a in range(0, N, 1024):
        x, t = s["x"][a:a + 1024].double(), s["targets"][a:a + 1024].long()
        z = torch.mm(x, w.t())
        if s["bias"] is not None:
            z += s["bias"].double()
        lses[a:a + 1024] = lse = torch.logsumexp(z, -1)
        rows = torch.nonzero((t >= 0) & (t < V))[:, 0]
        loss[a + rows] = lse[rows] - z[rows, t[rows]]
        if c["op"] == "grad":
            p = torch.softmax(z, -1)
            p[rows, t[rows]] -= 1
            gr = torch.zeros(x.shape[0], dtype=torch.float64, device="cuda")
            gr[rows] = s["grad"][a:a + 1024].double()[rows]
            p *= gr[:, None]
            dx[a:a + 1024] = torch.mm(p, w)
            dw += torch.mm(p.t().contiguous(), x)
            db += p.sum(0)
    if c["op"] == "loss":
        return {"loss": loss, "lse": lses}
    got = {"loss": loss, "dx": dx, "dw": dw}
    if s["bias"] is not None:
        got["dbias"] = db
    return got
