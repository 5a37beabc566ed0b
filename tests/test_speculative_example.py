"""The example model, whose every step runs the library's kernels, against the
same model written plainly in fp32 over whole sequences.

Tolerance: each of a layer's ten bf16 roundings is off by at most 2^-8 of its
value; over two layers and the head they add, as independent ones, to about
sqrt(22) 2^-8 / 2 = 1 % of the logits' norm; 5 % leaves room for how they grow
on the way.  Every expert is chosen (with fewer, a routing decision whose
logits nearly tie would fall differently here and there)."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def plain_logits(m, tokens):
    c = m.c
    rms = lambda x, w: x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
    x = m.embed[torch.tensor(tokens, device=m.device)].float()
    T = len(tokens)
    pos = torch.arange(T, device=m.device).double()
    angle = pos[:, None] * 10000.0 ** (-torch.arange(0, c.head_dim, 2, device=m.device).double() / c.head_dim)
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turned(v):
        a, b = v.chunk(2, -1)
        return torch.cat((a * cos - b * sin, a * sin + b * cos), -1)

    for w in m.weights:
        qkv = (rms(x, w["norm1"]) @ w["qkv"].float()).view(T, -1, c.head_dim)
        q, k, v = qkv.split([c.heads, c.kv_heads, c.kv_heads], 1)
        q, k = turned(rms(q, w["q_norm"])), turned(rms(k, w["k_norm"]))
        k, v = (t.repeat_interleave(c.heads // c.kv_heads, 1) for t in (k, v))
        s = torch.einsum("qhd,khd->hqk", q, k) * c.head_dim ** -0.5
        s = s.masked_fill(torch.ones(T, T, device=m.device).triu(1).bool(), float("-inf"))
        x = x + torch.einsum("hqk,khd->qhd", s.softmax(-1), v).flatten(1) @ w["out"].float()
        y = rms(x, w["norm2"])
        top, ids = (y @ w["router"].float().T).topk(c.topk, 1)
        weight = top.softmax(1)
        gu = torch.einsum("th,teih->tei", y, w["gate_up"][ids].float())
        g, u = gu.chunk(2, -1)
        x = x + torch.einsum("tei,tehi,te->th", torch.nn.functional.silu(g) * u, w["down"][ids].float(), weight)
    return rms(x, m.norm) @ m.head_weight.float().T


@pytest.fixture(scope="module")
def model():
    import speculative_decode as E
    m = E.Model(E.Config(experts=4, topk=4))
    yield m
    m.close()


def close(got, want):
    off = ((got - want).norm(dim=1) / want.norm(dim=1)).max().item()
    assert off < 0.05, off


def test_chunks_steps_forks_and_trees_match_the_plain_model(model):
    g = torch.Generator().manual_seed(3)
    tokens = torch.randint(0, model.c.vocab, (150,), generator=g).tolist()
    want = plain_logits(model, tokens)
    seq = model.cache.open()
    close(model.forward([seq], [tokens[:97]]), want[:97])      # a prompt's chunk
    close(model.forward([seq], [tokens[97:98]]), want[97:98])  # one token
    close(model.forward([seq], [tokens[98:104]]), want[98:104])  # a chain
    twin = model.cache.fork(seq)
    other = tokens[:104] + [7, 8, 9]
    got = model.forward([seq, twin], [tokens[104:110], [7, 8, 9]])  # both write after the fork
    close(got[:6], want[104:110])
    close(got[6:], plain_logits(model, other)[104:])
    # a tree below token 110: branches 111.. of the text and of other tokens
    n = model.cache.length(seq)
    branch = [1, 2, 3]
    tree = tokens[110:114] + branch
    seen = [1, 3, 7, 15, 1 | 16, 1 | 16 | 32, 1 | 16 | 32 | 64]
    words = torch.tensor(seen, dtype=torch.int64, device=model.device)
    got = model.forward([seq], [tree], positions=[n, n + 1, n + 2, n + 3, n + 1, n + 2, n + 3], tree_mask=words)
    close(got[:4], want[110:114])
    close(got[4:], plain_logits(model, tokens[:111] + branch)[111:])
    model.cache.keep(seq, n, [0, 4, 5])
    model.cache.free(twin)
    model.cache.compact()
    text = tokens[:111] + branch[:2] + [33, 44]
    close(model.forward([seq], [[33, 44]]), plain_logits(model, text)[-2:])
    model.cache.free(seq)
    assert model.cache.table.free_pages == model.c.pages and model.attention.status() == 0


def test_drafts_change_the_passes_only(model):
    import speculative_decode as E
    prompt = torch.randint(0, 50, (60,), generator=torch.Generator().manual_seed(4)).tolist()
    results = []
    for n in (0, 5):
        seq, tokens, passes = E.decode(model, prompt, steps=25, n_drafts=n, top_k=2, temperature=0.3)
        results.append((tokens, passes))
        model.cache.free(seq)
    (plain, one_each), (drafted, passes) = results
    assert one_each == 25 and passes <= one_each
    # the same draws, up to the first one whose logits nearly tie
    same = next((i for i, (a, b) in enumerate(zip(plain, drafted)) if a != b), len(plain))
    assert same > len(prompt)


def test_main_runs():
    import speculative_decode as E
    assert len(E.main()) == 170
