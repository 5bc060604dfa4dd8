"""Checks of the second pass that come before anything reaches the GPU."""
import pytest
import torch

from ctc_prefix_beam_amd import rescore


def model(vocab=32, max_len=6):
    return rescore.LanguageModel(rescore.ModelConfig(vocab=vocab, hidden=16, head_dim=8, layers=1,
                                                     max_len=max_len), device="cpu")


def nbest(lengths, L, label=3):
    lens = torch.tensor(lengths, dtype=torch.int32)
    at = torch.arange(L)
    tokens = torch.where(at < lens[..., None], label, -1).to(torch.int32)
    return tokens, lens


def test_hypotheses_longer_than_the_model_are_refused():
    """The model has positions 0 .. max_len: an index past them would be read on the GPU."""
    with pytest.raises(ValueError, match="max_len"):
        rescore.score(model(max_len=6), *nbest([[3, 7]], 10))
    with pytest.raises(ValueError, match="max_len"):
        rescore.train_output(model(max_len=6), *nbest([[7]], 10))


@pytest.mark.parametrize("label", [32, 1000])
def test_labels_outside_the_vocabulary_are_refused(label):
    with pytest.raises(ValueError, match="vocabulary"):
        rescore.score(model(vocab=32), *nbest([[3, 0]], 5, label=label))


def test_no_hypotheses():
    tokens, lens = nbest([[0] * 4], 5)
    got = rescore.score(model(), tokens[:0], lens[:0])
    assert got.shape == (0, 4)


def test_utterances():
    lp, lens = rescore.utterances(2, 30, 16, seed=3)
    assert lp.shape == (2, 30, 16) and lens.tolist() == [30, 30]
    assert (lp.exp().sum(-1) - 1).abs().max() < 1e-5
    assert (lp.argmax(-1) == 0).any() and (lp.argmax(-1) > 0).any()
