"""The quantised cache, the shared prefix and the adjusted logits together, as a
batch of answers uses them: the example model's steps against the same model
written plainly in fp32.

Tolerance: 5 % of the logits' norm for the roundings to 16 bits, as
test_speculative_example derives it.  Over codes the plain model holds its keys
and values as codes too; the 16-bit roundings before them (2^-8, some of them)
move a value across the border of two codes, 2^-4 apart at least, in at most one
case of eight, by at most 2^-3 of it: sqrt(1/8) 2^-3, 4.4 % more."""
import os
import sys

import pytest
import torch

from tests.test_quantised_cache import E4M3, exponent

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def held(x):
    """What a row's codes stand for."""
    e = exponent(x.abs().amax(-1))[..., None]
    return torch.ldexp(torch.ldexp(x, -e).clamp(-448, 448).to(E4M3).float(), e)


def plain_logits(m, tokens, codes):
    c = m.c
    rms = lambda x, w: x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
    x = m.embed[torch.tensor(tokens, device=m.device)].float()
    T = len(tokens)
    freq = 10000.0 ** (-torch.arange(0, c.head_dim, 2, device=m.device).double() / c.head_dim)
    angle = torch.arange(T, device=m.device).double()[:, None] * freq
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turned(v):
        a, b = v.chunk(2, -1)
        return torch.cat((a * cos - b * sin, a * sin + b * cos), -1)

    for w in m.weights:
        qkv = (rms(x, w["norm1"]) @ w["qkv"].float()).view(T, -1, c.head_dim)
        q, k, v = qkv.split([c.heads, c.kv_heads, c.kv_heads], 1)
        q, k = turned(rms(q, w["q_norm"])), turned(rms(k, w["k_norm"]))
        if codes:
            k, v = held(k), held(v)
        k, v = (t.repeat_interleave(c.heads // c.kv_heads, 1) for t in (k, v))
        s = torch.einsum("qhd,khd->hqk", q, k) * c.head_dim ** -0.5
        s = s.masked_fill(torch.ones(T, T, device=m.device).triu(1).bool(), float("-inf"))
        x = x + torch.einsum("hqk,khd->qhd", s.softmax(-1), v).flatten(1) @ w["out"].float()
        y = rms(x, w["norm2"])
        top, ids = (y @ w["router"].float().T).topk(c.topk, 1)
        weight = top.softmax(1)
        g, u = torch.einsum("th,teih->tei", y, w["gate_up"][ids].float()).chunk(2, -1)
        x = x + torch.einsum("tei,tehi,te->th", torch.nn.functional.silu(g) * u, w["down"][ids].float(), weight)
    return rms(x, m.norm) @ m.head_weight.float().T


@pytest.fixture(scope="module", params=[torch.bfloat16, E4M3], ids=["bf16", "codes"])
def model(request):
    import speculative_decode as E
    m = E.Model(E.Config(experts=4, topk=4, cache=request.param, pages=96))
    yield m
    m.close()


def close(model, got, want):
    off = ((got - want).norm(dim=1) / want.norm(dim=1)).max().item()
    assert off < (0.094 if model.c.cache == E4M3 else 0.05), off


def test_forks_of_a_prompt_match_the_plain_model(model):
    codes = model.c.cache == E4M3
    g = torch.Generator().manual_seed(3)
    prompt = torch.randint(0, model.c.vocab, (150,), generator=g).tolist()
    first = model.cache.open()
    close(model, model.forward([first], [prompt]), plain_logits(model, prompt, codes))
    seqs = [first] + [model.cache.fork(first) for _ in range(5)]
    made = [[] for _ in seqs]
    for step, lens in enumerate(([1] * 6, [1, 3, 2, 1, 6, 1], [1] * 6)):
        new = [torch.randint(0, model.c.vocab, (n,), generator=g).tolist() for n in lens]
        assert model.cache.shared_prefix(seqs) == 144
        logits = model.forward(seqs, new, share=True)
        for m, t in zip(made, new):
            m += t
        want = [plain_logits(model, prompt + m, codes)[-n:] for m, n in zip(made, lens)]
        close(model, logits, torch.cat(want))
    for s in seqs:
        model.cache.free(s)
    assert model.cache.table.free_pages == model.c.pages and model.attention.status() == 0


def test_answers_follow_the_grammar_and_the_penalties(model):
    import batched_answers as B
    prompt = list(range(40, 100))
    letters, digits = list(range(0, 600, 3)), [601, 777, 999]
    grammar = lambda answer: digits if len(answer) % 3 == 2 else letters
    seqs, made = B.answers(model, prompt, n=4, steps=9, allowed=grammar, biases=[(0, -1e9), (3, 4.0)])
    for m in made:
        assert len(m) == 9 and all(t in grammar(m[:i]) for i, t in enumerate(m)) and 0 not in m
    for s in seqs:
        model.cache.free(s)
    # what has been said costs more than any logit gives: no token twice
    seqs, made = B.answers(model, prompt, n=3, steps=20, repetition=1.0, presence=1e4, frequency=0.0)
    assert all(len(set(m)) == 20 for m in made)
    for s in seqs:
        model.cache.free(s)
    assert model.cache.table.free_pages == model.c.pages and model.attention.status() == 0


def test_main_runs():
    import batched_answers as B
    made = B.main()
    assert len(made) == 5 and all(t % 2 == i % 2 for m in made for i, t in enumerate(m))
