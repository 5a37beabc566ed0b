"""Decoding with drafts draws what the model says: with drafts that are all
right, wrong at some place or none, each token is the plain model's greedy
choice after the tokens before it, right drafts save their passes, and the cache
holds what the next token needs.

Tolerance: the logits of a row are within 5 % of its norm (as in
test_speculative_example), so one of them by about 5 % of the row's root mean
square, by four times that at most; a token is the greedy choice if its plain
logit is within twice that, 0.4 of the root mean square, of the largest (which
of 1000 random tokens two or three are)."""
import os
import sys

import pytest
import torch

from tests.test_speculative_example import close, plain_logits

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
STEPS = 25


@pytest.fixture(scope="module")
def model():
    import speculative_decode as E
    m = E.Model(E.Config(experts=4, topk=4), seed=1)
    yield m
    m.close()


@pytest.fixture(scope="module")
def prompt(model):
    return torch.randint(0, model.c.vocab, (61,), generator=torch.Generator().manual_seed(5)).tolist()


def off(row, token):
    """How far a token is from being the greedy choice, in root mean squares."""
    return float((row.max() - row[token]) / row.square().mean().sqrt())


def decode(model, prompt, n_drafts):
    import speculative_decode as E
    seq, tokens, passes = E.decode(model, prompt, steps=STEPS, n_drafts=n_drafts, temperature=0.0, top_k=0, top_p=1.0)
    assert len(tokens) == len(prompt) + STEPS
    want = plain_logits(model, tokens)
    for p in range(len(prompt), len(tokens)):
        assert off(want[p - 1], tokens[p]) <= 0.4, f"position {p}"
    return seq, tokens, passes, want


@pytest.fixture(scope="module")
def greedy(model, prompt):
    seq, tokens, passes, _ = decode(model, prompt, 0)
    model.cache.free(seq)
    assert passes == STEPS
    return tokens


# (drafts of a pass, the one that is wrong): tokens of a pass are those before it and the model's own
@pytest.mark.parametrize("n,wrong", [(5, None), (5, 2), (5, 0), (3, 2), (1, None), (7, 5), (11, None)])
def test_drafts_are_kept_up_to_the_first_wrong_one(model, prompt, greedy, monkeypatch, n, wrong):
    import speculative_decode as E
    given = []

    def draft(history, most):
        assert most == n
        drafts = greedy[len(history):len(history) + n]
        if wrong is not None and len(drafts) > wrong:
            drafts[wrong] = (drafts[wrong] + 1) % model.c.vocab
        given.append(drafts)
        return drafts

    monkeypatch.setattr(E, "draft", draft)
    seq, tokens, passes, want = decode(model, prompt, n)
    assert any(given) and passes < STEPS or wrong == 0
    same = next((i for i, (a, b) in enumerate(zip(greedy, tokens)) if a != b), len(tokens))
    if same < len(tokens):  # two tokens that nearly tie
        assert same >= len(prompt) and off(want[same - 1], greedy[same]) <= 0.4
    else:
        each = n + 1 if wrong is None else wrong + 1
        assert passes == 1 + -(-(STEPS - 1) // each)
        if (STEPS - 1) % each == 0:
            # the cache ends before the last token, and goes on from there
            assert model.cache.length(seq) == len(tokens) - 1
            close(model.forward([seq], [tokens[-1:]]), want[-1:])
    model.cache.free(seq)
    assert model.cache.table.free_pages == model.c.pages and model.attention.status() == 0


def test_drafts_by_lookup(model, prompt):
    import speculative_decode as E
    text = list(range(50))
    assert E.draft(text + [10], 3) == [11, 12, 13] and E.draft(text + text + [48], 5) == [49, 48]
    assert E.draft(text, 5) == []
    seq, _, passes, _ = decode(model, prompt[:20] * 3, 5)
    assert passes <= STEPS
    model.cache.free(seq)
