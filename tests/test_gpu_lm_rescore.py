"""The second pass over N-best lists: scores through the paged cache against the
same model run densely in float64, and training of its output layer."""
import numpy as np
import pytest
import torch

import ctc_prefix_beam_amd as cpb
import synth
from ctc_prefix_beam_amd import rescore

pytestmark = pytest.mark.gpu


def nbest(V=64, T=60, B=3, N=4):
    lp, lens = synth.peaky(B, T, V, seed=1, p_blank=0.5, lengths=(T // 3, T))
    dec = cpb.OfflineDecoder(cpb.DecoderConfig(beam=N, nbest=N, blank_threshold=1.0, max_out_len=T))
    return dec.decode(torch.from_numpy(lp).cuda(), torch.from_numpy(lens).cuda())


def dense(model, tokens):
    """Log-probability of one hypothesis (a list of labels), all in float64 on the CPU."""
    c = model.cfg
    f = lambda a: a.cpu().double()   # noqa: E731

    def norm(x):
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    ids = torch.tensor([0] + tokens)
    n = len(ids)
    x = f(model.embed)[ids] + f(model.position)[:n]
    mask = torch.ones((n, n), dtype=torch.bool).tril()
    for i in range(c.layers):
        qkv = (norm(x) @ f(model.qkv[i]).t()).view(n, -1, c.head_dim)
        q, k, v = qkv.split((c.q_heads, c.kv_heads, c.kv_heads), 1)
        g = c.q_heads // c.kv_heads
        heads = []
        for h in range(c.q_heads):
            s = q[:, h] @ k[:, h // g].t() / c.head_dim ** 0.5
            p = torch.softmax(torch.where(mask, s, -torch.inf), -1)
            heads.append(p @ v[:, h // g])
        x = x + torch.cat(heads, -1) @ f(model.o[i]).t()
        x = x + torch.nn.functional.gelu(norm(x) @ f(model.up[i]).t()) @ f(model.down[i]).t()
    z = norm(x) @ f(model.out).t() + f(model.bias)
    z = z - torch.logsumexp(z, -1, keepdim=True)
    return float(z[torch.arange(n), torch.tensor(tokens + [0])].sum())


def test_scores_equal_the_dense_model():
    tokens, lengths, _ = nbest()
    model = rescore.LanguageModel(rescore.ModelConfig(vocab=64, hidden=64, head_dim=32,
                                                      max_len=80, dtype=torch.float32))
    got = rescore.score(model, tokens, lengths)
    assert len(set(lengths.flatten().tolist())) > 1
    for b in range(tokens.shape[0]):
        for n in range(tokens.shape[1]):
            hyp = tokens[b, n, :int(lengths[b, n])].tolist()
            want = dense(model, hyp)
            # float32 products of 64 terms through two layers, summed over the tokens
            assert abs(float(got[b, n]) - want) <= 2.0 ** -16 * (len(hyp) + 1) * 8


def test_a_cache_with_fewer_pages_scores_the_same():
    tokens, lengths, _ = nbest()
    model = rescore.LanguageModel(rescore.ModelConfig(vocab=64, hidden=64, head_dim=32, max_len=80))
    want = rescore.score(model, tokens, lengths)
    pages = int(((lengths + 1 + 15) // 16).sum())   # what the hypotheses need, and not one more
    full = model.cache
    model.cache = lambda rows, max_len: full(rows, max_len, pages)
    assert torch.equal(rescore.score(model, tokens, lengths), want)


def test_training_lowers_the_loss_and_moves_the_order():
    tokens, lengths, scores = nbest()
    model = rescore.LanguageModel(rescore.ModelConfig(vocab=64))
    before = rescore.score(model, tokens, lengths)
    losses = rescore.train_output(model, tokens[:, :1], lengths[:, :1], steps=20)
    assert torch.isfinite(losses).all() and losses[-1] < 0.7 * losses[0]
    after = rescore.score(model, tokens, lengths)
    assert (after[:, 0] > before[:, 0]).all()
    order, combined = rescore.rescore(model, tokens, lengths, scores, weight=1.0)
    c = np.take_along_axis(combined.cpu().numpy(), order.cpu().numpy(), 1)
    assert (np.diff(c, axis=1) <= 0).all()
