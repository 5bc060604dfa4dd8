"""The second pass in 8 bits: the operators in a row, as the model calls them, each against
64 bits on what it was given; captured steps."""
import math

import numpy as np
import pytest
import torch

import ctc_prefix_beam_amd as cpb
import lm_ref
import lm_ref8
import synth
from ctc_prefix_beam_amd import lm, rescore

pytestmark = pytest.mark.gpu
CODES = [torch.int8, torch.float8_e4m3fn]


def nbest(V=64, T=40, B=2, N=3):
    lp, lens = synth.peaky(B, T, V, seed=1, p_blank=0.5, lengths=(T // 3, T))
    dec = cpb.OfflineDecoder(cpb.DecoderConfig(beam=N, nbest=N, blank_threshold=1.0, max_out_len=T))
    return dec.decode(torch.from_numpy(lp).cuda(), torch.from_numpy(lens).cuda())


def config(code, dtype, **kw):
    return rescore.ModelConfig(**{**dict(vocab=64, hidden=64, head_dim=32, max_len=80, dtype=dtype,
                                         cache_dtype=code, weights8=True), **kw})


class Checked:
    """The operators with a check of each call, on the inputs that it had."""

    def __init__(self, monkeypatch):
        self.calls = {}
        for name in ("linear8", "cache_store8", "attention8"):
            monkeypatch.setattr(lm, name, self.around(name, getattr(lm, name)))

    def around(self, name, f):
        def call(*a, **kw):
            self.calls[name] = self.calls.get(name, 0) + 1
            return getattr(self, name)(f, *a, **kw)
        return call

    def linear8(self, f, x, w, ws):
        out = f(x, w, ws)
        want, tol = lm_ref8.linear(*lm_ref8.quantize(x), w, ws, None, x.dtype)
        assert ((out.cpu().double() - want).abs() <= tol).all()
        return out

    def cache_store8(self, f, k, v, slots, kc, vc, ks, vs, stream=None):
        want = lm_ref8.store(k, slots, kc, ks), lm_ref8.store(v, slots, vc, vs)
        f(k, v, slots, kc, vc, ks, vs, stream)
        held = torch.zeros(kc.shape[:2], dtype=torch.bool)
        held.view(-1)[slots.cpu().long()[slots.cpu() >= 0]] = True
        for (values, scales), c, s in zip(want, (kc, vc), (ks, vs)):
            assert torch.equal(s.cpu().double(), scales)
            assert torch.equal(lm_ref8.values(c)[held], values[held])

    def attention8(self, f, q, kc, vc, ks, vs, tables, lens, *a, **kw):
        out, lse = f(q, kc, vc, ks, vs, tables, lens, *a, **kw)
        real = [lm_ref8.values(c) * s.cpu().double()[:, None, :, None] for c, s in ((kc, ks), (vc, vs))]
        wo, wl, to, tl = lm_ref.attention(q, *real, tables, lens, q.shape[2] ** -0.5, 0, kc.shape[1])
        assert ((out.cpu().double() - wo).abs() <= to).all()
        dead = wl == -math.inf
        assert ((lse.cpu().double() - wl).abs()[~dead] <= tl[~dead]).all()
        return out, lse


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_every_call_of_the_model(code, dtype, monkeypatch):
    tokens, lengths, _ = nbest()
    model = rescore.LanguageModel(config(code, dtype))
    checked = Checked(monkeypatch)
    got = rescore.score(model, tokens, lengths)
    assert torch.isfinite(got).all() and (got < 0).all()
    steps = int(lengths.max()) + 1
    assert checked.calls == {"linear8": 8 * steps, "cache_store8": 2 * steps,
                             "attention8": 2 * steps}


def test_only_the_cache_or_only_the_weights():
    tokens, lengths, _ = nbest()
    for cfg in (config(None, torch.bfloat16), config(torch.int8, torch.float16, weights8=False)):
        model = rescore.LanguageModel(cfg)
        assert isinstance(model.up[0], torch.Tensor) != cfg.weights8
        assert (model.cache(2, 20).k.dtype == torch.int8) == (cfg.cache_dtype is not None)
        assert torch.isfinite(rescore.score(model, tokens, lengths)).all()
    eight = rescore.in_8_bits(rescore.ModelConfig(vocab=9))
    assert eight.weights8 and eight.cache_dtype == torch.int8 and eight.vocab == 9


def test_a_cache_with_fewer_pages_scores_the_same():
    tokens, lengths, _ = nbest()
    model = rescore.LanguageModel(config(torch.int8, torch.bfloat16))
    want = rescore.score(model, tokens, lengths)
    pages = int(((lengths + 1 + 15) // 16).sum())   # what the hypotheses need, and not one more
    full = model.cache
    model.cache = lambda rows, max_len: full(rows, max_len, pages)
    assert torch.equal(rescore.score(model, tokens, lengths), want)


def test_training_and_rescoring_run():
    tokens, lengths, scores = nbest()
    model = rescore.LanguageModel(config(torch.int8, torch.bfloat16))
    losses = rescore.train_output(model, tokens[:, :1], lengths[:, :1], steps=3)
    assert torch.isfinite(losses).all()
    order, combined = rescore.rescore(model, tokens, lengths, scores)
    c = np.take_along_axis(combined.cpu().numpy(), order.cpu().numpy(), 1)
    assert (np.diff(c, axis=1) <= 0).all()


def test_the_example_in_8_bits(capsys):
    rescore.main(bits=8)
    lines = capsys.readouterr().out.splitlines()
    assert [l.split(":")[0] for l in lines] == ["order before training", "loss per token",
                                                "order after training",
                                                "best of the first utterance"]


@pytest.mark.parametrize("code", CODES)
def test_pages_handed_on_begin_anew(code):
    """A request's pages go to another one, whose values are far smaller: nothing of the old scales
    stays.  What is read back is as near as the new values' own scale says."""
    c = lm.PagedCache(2, 64, 2, 32, code, page_size=8, num_pages=8)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")   # noqa: E731
    big = torch.randn((60, 2, 32), device="cuda") * 1000
    c.store(big, -big, c.append(i32(60, 0), 60).slots)
    c.release(torch.tensor([1, 0], dtype=torch.uint8, device="cuda"))
    small = torch.randn((50, 2, 32), device="cuda") * 0.001
    plan = c.append(i32(0, 50), 50)
    assert not plan.status.any()
    c.store(small, -small, plan.slots)
    k, v = c.load(plan.slots, dtype=torch.float32)
    step = 2 * float(small.abs().max()) / lm_ref8.TOP[code]   # above the scale of any page
    near = step / 2 if code == torch.int8 else step * 16      # e4m3: half a step of 32 at the top
    assert ((k - small).abs() <= near).all() and torch.equal(v, -k)
    out, _ = c.attend(torch.zeros((2, 2, 32), device="cuda"))
    want = v.cpu().double().mean(0)
    assert ((out[1].cpu().double() - want).abs() <= 2.0 ** -16 * float(v.abs().max())).all()
    with pytest.raises(ValueError):
        lm.PagedCache(1, 16, 1, 32).load(plan.slots[:1])


def test_a_captured_step_is_replayed_for_one_token_after_another():
    """Plan, projection, store, attention and projection in one graph."""
    rows, heads, D, H, steps = 3, 2, 64, 96, 40
    g = torch.Generator(device="cuda").manual_seed(4)
    inputs = torch.randn((steps, rows, H), generator=g, device="cuda").to(torch.bfloat16)
    wi = lm.quantize_rows(torch.randn((3 * heads * D, H), generator=g, device="cuda"))
    wo = lm.quantize_rows(torch.randn((H, heads * D), generator=g, device="cuda"))
    ones = torch.ones(rows, dtype=torch.int32, device="cuda")

    def cache():
        c = lm.PagedCache(rows, 64, heads, D, torch.int8)
        c.append(torch.tensor([0, 3, 7], dtype=torch.int32, device="cuda"), 10)
        c.k.zero_()
        c.v.zero_()
        return c

    def step(c, x):
        plan = lm.cache_plan(c.lengths, ones, c.tables, c.pool, c.taken, c.page_size, rows)
        q, k, v = lm.linear8(x, *wi).view(rows, 3, heads, D).unbind(1)
        c.store(k, v, plan.slots)
        out, lse = lm.attention8(q, *c._codes(0), c.tables, plan.lengths)
        y = lm.linear8(out.reshape(rows, -1), *wo)
        c.lengths.copy_(plan.lengths)
        c.taken.copy_(plan.taken)
        return y, lse
    a, b, x = cache(), cache(), torch.empty_like(inputs[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(a, x)
    for i in range(steps):
        x.copy_(inputs[i])
        graph.replay()
        want = step(b, inputs[i])
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), i
        assert torch.equal(a.k, b.k) and torch.equal(a.k_scale, b.k_scale), i
        assert torch.equal(a.v_scale, b.v_scale), i
    assert a.lengths.tolist() == [steps, steps + 3, steps + 7]
