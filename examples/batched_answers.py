"""Several answers to one prompt, decoded as a batch of forks on an E4M3 cache:
the prompt goes in once and its pages are read once a step for all answers,
repeated tokens are penalised, some tokens biased, and a grammar says which may
follow.

    python examples/batched_answers.py

The model is the small one of speculative_decode.py.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from speculative_decode import Config, Model
from weight_streaming_expert_gb300 import adjust_logits, sample


def mask_of(allowed, vocab, device):
    """A row of a grammar's mask: a bit for each token that may follow."""
    words = [0] * -(-vocab // 32)
    for t in allowed:
        words[t // 32] |= 1 << (t % 32)
    return torch.tensor([w - (1 << 32) if w >> 31 else w for w in words], dtype=torch.int32, device=device)


def answers(model, prompt, n, steps, seed=0, temperature=0.9, top_k=50, repetition=1.2, presence=0.2, frequency=0.1,
            biases=(), allowed=None):
    """`n` answers of `steps` tokens each to the prompt.  biases: (token, bias)
    pairs; allowed(answer): the tokens that may follow an answer (a list), None:
    all.  Returns (their sequences, the answers)."""
    device, vocab = model.device, model.c.vocab
    u = torch.rand(steps, n, generator=torch.Generator().manual_seed(seed)).to(device)
    full = lambda v, dt=torch.float32: torch.full((n,), v, dtype=dt, device=device)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=device)
    settings = dict(repetition=full(repetition), presence=full(presence), frequency=full(frequency))
    if biases:
        settings.update(bias_ids=i32([t for t, _ in biases] * n),
                        bias_values=torch.tensor([b for _, b in biases] * n, device=device),
                        bias_starts=i32([i * len(biases) for i in range(n + 1)]))
    first = model.cache.open()
    logits = model.forward([first], [prompt])[-1:].expand(n, -1)
    seqs = [first] + [model.cache.fork(first) for _ in range(n - 1)]
    made = [[] for _ in range(n)]
    for step in range(steps):
        history, spans = [], []
        for m in made:  # the prompt, and each answer so far
            spans.append([len(history), len(history) + len(prompt), len(history) + len(prompt) + len(m)])
            history += prompt + m
        mask = None
        if allowed is not None:
            mask = torch.stack([mask_of(allowed(m), vocab, device) for m in made])
        logits = adjust_logits(logits, history=i32(history), spans=i32(spans), allowed=mask, **settings)
        tokens = sample(logits, u[step], full(temperature), full(top_k, torch.int32)).tolist()
        for m, t in zip(made, tokens):
            m.append(t)
        if step + 1 < steps:
            logits = model.forward(seqs, [[t] for t in tokens], share=True)
    return seqs, made


def main():
    model = Model(Config(cache=torch.float8_e4m3fn))
    prompt = torch.randint(0, model.c.vocab, (90,), generator=torch.Generator().manual_seed(1)).tolist()
    even = list(range(0, model.c.vocab, 2))
    odd = list(range(1, model.c.vocab, 2))
    seqs, made = answers(model, prompt, n=5, steps=12, biases=[(0, -5.0), (7, 2.0)],
                         allowed=lambda answer: odd if len(answer) % 2 else even)  # a grammar of turns
    for m in made:
        print(m)
    held = model.c.pages - model.cache.table.free_pages
    print(f"{held} pages of {model.c.page} positions hold {len(seqs)} sequences of {model.cache.length(seqs[0])}")
    assert model.attention.status() == 0
    model.close()
    return made


if __name__ == "__main__":
    main()
