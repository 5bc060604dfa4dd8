"""Second pass over N-best lists: a language model scores every hypothesis of the
decoder token by token, with a paged key/value cache, and its output layer is
trained on the best ones.

    python -m ctc_prefix_beam_amd.rescore

decodes seeded synthetic utterances, rescores their 8-best lists with a small
randomly initialised model, takes training steps on its output layer with the
first-pass best hypotheses as targets, and rescores again.  It runs the
operators of ``ctc_prefix_beam_amd.lm`` together as a user would: pages and
slots from the hypotheses' lengths (of which only the longest is read back), the
store of new keys and values, attention over the cache, and token losses with
gradients.
Projections and normalisations are plain torch.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import lm


@dataclass
class ModelConfig:
    vocab: int
    layers: int = 2
    hidden: int = 256
    q_heads: int = 4
    kv_heads: int = 2
    head_dim: int = 64
    max_len: int = 1024
    dtype: torch.dtype = torch.bfloat16


class LanguageModel:
    """A decoder-only model; label 0 (the decoder's blank) begins and ends a
    hypothesis."""

    def __init__(self, cfg: ModelConfig, seed: int = 0, device="cuda"):
        self.cfg = c = cfg
        g = torch.Generator().manual_seed(seed)

        def weight(rows, cols):
            return (torch.randn((rows, cols), generator=g) / cols ** 0.5).to(c.dtype).to(device)
        self.embed = weight(c.vocab, c.hidden)
        self.position = weight(c.max_len + 1, c.hidden)
        heads = c.q_heads + 2 * c.kv_heads
        self.qkv = [weight(heads * c.head_dim, c.hidden) for _ in range(c.layers)]
        self.o = [weight(c.hidden, c.q_heads * c.head_dim) for _ in range(c.layers)]
        self.up = [weight(4 * c.hidden, c.hidden) for _ in range(c.layers)]
        self.down = [weight(c.hidden, 4 * c.hidden) for _ in range(c.layers)]
        self.out = weight(c.vocab, c.hidden)
        self.bias = torch.zeros(c.vocab, device=device)

    def cache(self, rows: int, max_len: int, num_pages: int = 0, page_size: int = 16):
        c = self.cfg
        return lm.PagedCache(rows, max_len, c.kv_heads, c.head_dim, c.dtype, page_size, num_pages,
                             self.embed.device, layers=c.layers)

    def step(self, tokens, alive, cache, max_len: int = 0):
        """Hidden states (rows, hidden) after one more token of every row with
        alive[r] (bool); the others' are not meaningful.  tokens: (rows,) int64.
        `max_len`: what no row holds more tokens than afterwards, where that is known
        (0: what the cache can hold)."""
        c, rows = self.cfg, tokens.numel()
        before = cache.lengths
        plan = cache.append(alive.to(torch.int32), rows)
        # one new token a row at most: its slot, or -1
        at = plan.starts[:-1].clamp(max=rows - 1).long()
        slots = torch.where(alive, plan.slots[at], -1)
        x = self.embed[tokens] + self.position[before.long()]
        for i in range(c.layers):
            qkv = (_norm(x) @ self.qkv[i].t()).view(rows, -1, c.head_dim)
            q, k, v = qkv.split((c.q_heads, c.kv_heads, c.kv_heads), 1)
            cache.store(k, v, slots, layer=i)
            a, _ = cache.attend(q, layer=i, max_len=max_len)
            x = x + a.reshape(rows, -1) @ self.o[i].t()
            x = x + torch.nn.functional.gelu(_norm(x) @ self.up[i].t()) @ self.down[i].t()
        return _norm(x)


def _norm(x):
    f = x.float()
    return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


def _longest(model: LanguageModel, toks, lens) -> int:
    """Tokens of the longest hypothesis (-1: there is none).  What the model's tables cannot
    be indexed with is refused here: on the GPU it would be read past their ends."""
    rows, L = toks.shape
    if rows == 0:
        return -1
    used = torch.arange(L, device=toks.device) < lens[:, None]
    label = torch.where(used, toks, -1).amax(1) if L else torch.full_like(lens, -1)
    longest, label = torch.stack((lens.clamp(max=L).amax(), label.amax())).tolist()
    if longest > model.cfg.max_len:
        raise ValueError(f"a hypothesis has {longest} tokens, the model's max_len is "
                         f"{model.cfg.max_len}")
    if label >= model.cfg.vocab:
        raise ValueError(f"label {label} is outside the model's vocabulary of {model.cfg.vocab}")
    return longest


def score(model: LanguageModel, tokens, lengths, keep_states: bool = False):
    """Log-probabilities (B, N) of hypotheses as the decoder gives them: tokens
    (B, N, L) int32, -1 padded, lengths (B, N) int32.  Each is scored with the end
    label after its last token (a hypothesis cut at L tokens without it).  With
    `keep_states`, also the (positions, rows, hidden) states and the (positions,
    rows) targets, -1 where a row has none."""
    B, N, L = tokens.shape
    rows = B * N
    toks, lens = tokens.reshape(rows, L), lengths.reshape(rows)
    longest = _longest(model, toks, lens)
    cache = model.cache(rows, L + 1)
    total = torch.zeros(rows, device=tokens.device)
    end = torch.zeros(rows, dtype=torch.int32, device=tokens.device)
    states, targets = [], []
    now = end.long()
    for t in range(longest + 1):
        alive = lens >= t
        target = toks[:, t] if t < L else torch.full_like(end, -1)
        target = torch.where(lens > t, target, torch.where(lens == t, end, -1)).contiguous()
        h = model.step(now, alive, cache, t + 1)
        loss, _ = lm.token_loss_forward(h, model.out, target, model.bias)
        total -= loss
        if keep_states:
            states.append(h)
            targets.append(target)
        now = target.clamp(min=0).long()
    total = total.view(B, N)
    if not keep_states:
        return total
    if not states:
        return total, model.out[:0][None], end[None]
    return total, torch.stack(states), torch.stack(targets)


def rescore(model: LanguageModel, tokens, lengths, scores, weight: float = 0.3):
    """(order (B, N), combined scores (B, N)): first-pass score plus `weight`
    times the model's, hypotheses in descending order (ties: the lower slot)."""
    combined = scores + weight * score(model, tokens, lengths)
    return torch.sort(combined, dim=1, descending=True, stable=True)[1], combined


def train_output(model: LanguageModel, tokens, lengths, steps: int = 10, rate: float = 1.0):
    """Gradient steps on the output layer for the given hypotheses (mean loss per
    token); returns the losses."""
    _, states, targets = score(model, tokens, lengths, keep_states=True)
    x, t = states.flatten(0, 1), targets.flatten()
    count = (t >= 0).sum().clamp(min=1)
    w, b = model.out.float(), model.bias
    losses = []
    for _ in range(steps):
        wd = w.to(model.cfg.dtype).requires_grad_()
        bd = b.clone().requires_grad_()
        loss = lm.token_loss(x, wd, t, bd).sum() / count
        loss.backward()
        w, b = w - rate * wd.grad.float(), b - rate * bd.grad
        losses.append(loss.detach())
    model.out, model.bias = w.to(model.cfg.dtype), b
    return torch.stack(losses)


def utterances(rows: int, frames: int, vocab: int, seed: int = 0):
    """Log-probabilities (rows, frames, vocab) as an acoustic model leaves them, a blank or
    another label ahead in each frame, and their lengths (rows,) int32, on the CPU."""
    g = torch.Generator().manual_seed(seed)
    z = torch.randn((rows, frames, vocab), generator=g)
    ahead = torch.randint(1, vocab, (rows, frames), generator=g)
    ahead[torch.rand((rows, frames), generator=g) < 0.6] = 0
    z.scatter_add_(2, ahead[..., None], torch.where(ahead == 0, 8.0, 6.0)[..., None])
    return z.log_softmax(-1), torch.full((rows,), frames, dtype=torch.int32)


def main():
    from . import DecoderConfig, OfflineDecoder
    lp, lens = utterances(8, 200, 256)
    dec = OfflineDecoder(DecoderConfig(beam=8, nbest=8, blank_threshold=0.999, max_out_len=100))
    tokens, lengths, scores = dec.decode(lp.cuda(), lens.cuda())
    model = LanguageModel(ModelConfig(vocab=256))
    order, _ = rescore(model, tokens, lengths, scores)
    print("order before training:", order[0].tolist())
    losses = train_output(model, tokens[:, :1], lengths[:, :1])
    print("loss per token:", " ".join(f"{v:.3f}" for v in losses.tolist()))
    order, combined = rescore(model, tokens, lengths, scores)
    print("order after training: ", order[0].tolist())
    best = int(order[0, 0])
    print("best of the first utterance:", tokens[0, best, :int(lengths[0, best])].tolist())


if __name__ == "__main__":
    main()
