"""A small model decoded with drafts, every step of it on the library's kernels:
queries and keys are normed and rotated on their way into the paged cache,
attention runs over the cache, the routed experts follow, and the vocabulary
projection's logits are sampled.  (The projections around attention and the
layer norms are plain torch.)

    python examples/speculative_decode.py

The prompt goes in as one chunk.  Each step then drafts tokens by looking up
what followed the last token before, verifies them as a chain, keeps those that
the model would have drawn and drops the rest from the cache.  At the end the
sequence is forked, the two continuations are drawn with different random
numbers, a tree of drafts is verified, and the cache is compacted.
"""
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from weight_streaming_expert_gb300 import LmHead, MoELayer, PagedAttention, PagedKVCache, QKNormRope, sample
from weight_streaming_expert_gb300.native import MOE_LM_HEAD_MAX_TOKENS, MOE_MAX_TOKENS


@dataclass
class Config:
    vocab: int = 1000
    hidden: int = 256
    layers: int = 2
    heads: int = 8
    kv_heads: int = 2
    head_dim: int = 64
    experts: int = 16
    topk: int = 2
    inter: int = 128
    page: int = 16
    pages: int = 64
    max_len: int = 512
    cache: torch.dtype = torch.bfloat16  # or float8_e4m3fn: quantised keys and values


def rms(x, w, eps=1e-6):
    y = x.float()
    return (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + eps) * w.float()).to(x.dtype)


class Model:
    def __init__(self, c: Config, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        rand = lambda *s, std=0.02: (torch.randn(*s, generator=g, device=device) * std).bfloat16()
        self.c, self.device = c, device
        self.embed = rand(c.vocab, c.hidden, std=1.0)
        width = (c.heads + 2 * c.kv_heads) * c.head_dim
        self.weights = []
        for _ in range(c.layers):
            self.weights.append(dict(
                norm1=1 + rand(c.hidden, std=0.1), norm2=1 + rand(c.hidden, std=0.1),
                qkv=rand(c.hidden, width, std=0.08),
                out=rand(c.heads * c.head_dim, c.hidden, std=0.08), q_norm=1 + rand(c.head_dim, std=0.1),
                k_norm=1 + rand(c.head_dim, std=0.1), router=rand(c.experts, c.hidden, std=0.1),
                gate_up=rand(c.experts, 2 * c.inter, c.hidden, std=0.08),
                down=rand(c.experts, c.hidden, c.inter, std=0.08)))
        self.norm = 1 + rand(c.hidden, std=0.1)
        self.head_weight = rand(c.vocab, c.hidden, std=0.15)
        self.moe = [MoELayer(w["router"], w["gate_up"], w["down"], c.topk) for w in self.weights]
        self.head = LmHead(self.head_weight)
        self.rope = QKNormRope(c.head_dim, device=device)
        self.attention = PagedAttention(c.heads, c.kv_heads, c.head_dim, device=device)
        self.cache = PagedKVCache(c.layers, c.pages, c.page, c.kv_heads, c.head_dim, c.max_len, dtype=c.cache,
                                  device=device)

    def forward(self, seqs, tokens, positions=None, tree_mask=None, share=False):
        """`tokens[b]`: the new tokens of sequence seqs[b], which enter the
        cache.  With `share` what forks have in common is read once for all of
        them.  Returns the fp32 logits of all tokens, one row each."""
        c, cache = self.c, self.cache
        lens = [len(t) for t in tokens]
        starts = [0]
        for n in lens:
            starts.append(starts[-1] + n)
        if positions is None:
            positions = [p for s, n in zip(seqs, lens) for p in range(cache.length(s), cache.length(s) + n)]
        slots = torch.cat([cache.extend(s, n) for s, n in zip(seqs, lens)])
        table, kv_lens = cache.block_table(seqs)
        prefix = cache.shared_prefix(seqs, max(lens)) if share else 0
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=self.device)
        positions, starts = i32(positions), i32(starts)
        x = self.embed[torch.tensor([t for ts in tokens for t in ts], device=self.device)]
        T, H, K, D = x.shape[0], c.heads, c.kv_heads, c.head_dim
        for layer, w in enumerate(self.weights):
            qkv = (rms(x, w["norm1"]) @ w["qkv"]).view(T, H + 2 * K, D)
            q = self.rope(qkv[:, :H], qkv[:, H:H + K], qkv[:, H + K:], w["q_norm"], w["k_norm"], positions, slots,
                          **cache.layer(layer))
            o = self.attention(q, block_table=table, q_starts=starts, kv_lens=kv_lens, max_q_len=max(lens),
                               tree_mask=tree_mask, prefix_len=prefix, **cache.layer(layer))
            x = x + o.view(T, H * D) @ w["out"]
            y = rms(x, w["norm2"])
            x = x + torch.cat([self.moe[layer](part)[0] for part in y.split(MOE_MAX_TOKENS)])
        return torch.cat([self.head(part.contiguous()) for part in rms(x, self.norm).split(MOE_LM_HEAD_MAX_TOKENS)])

    def close(self):
        for layer in self.moe:
            layer.close()
        self.head.close()
        self.attention.close()


def draft(history, n):
    """What followed the last token where it stood before, up to n tokens."""
    for i in range(len(history) - 2, -1, -1):
        if history[i] == history[-1]:
            return history[i + 1:i + 1 + n]
    return []


def decode(model, prompt, steps, n_drafts, seed=0, temperature=0.8, top_k=20, top_p=0.95):
    """Draws `steps` tokens after the prompt; position p uses random number
    u[p], whether it was drafted or not, so the drafts change the number of
    passes and nothing else.  Returns (sequence, its tokens, passes)."""
    device = model.device
    u = torch.rand(model.c.max_len + n_drafts + 1, generator=torch.Generator().manual_seed(seed)).to(device)

    def draw(logits, first):  # the tokens at positions first, first + 1, ..
        n = logits.shape[0]
        full = lambda v, dt: torch.full((n,), v, dtype=dt, device=device)
        return sample(logits, u[first:first + n], full(temperature, torch.float32), full(top_k, torch.int32),
                      full(top_p, torch.float32)).tolist()

    seq = model.cache.open()
    tokens = list(prompt)
    tokens += draw(model.forward([seq], [tokens])[-1:], len(tokens))
    passes = 1
    while len(tokens) < len(prompt) + steps:
        at = len(tokens) - 1  # the last token is not in the cache yet
        drafts = draft(tokens, n_drafts)
        drawn = draw(model.forward([seq], [[tokens[-1]] + drafts]), at + 1)
        passes += 1
        good = 0
        while good < len(drafts) and drafts[good] == drawn[good]:
            good += 1
        tokens += drawn[:good + 1]
        model.cache.truncate(seq, at + 1 + good)  # the rejected drafts leave the cache
    return seq, tokens[:len(prompt) + steps], passes


def verify_tree(model, seq, root, branches):
    """Verifies drafts that branch after `root`: each branch is a chain.
    Greedy; returns the accepted tokens, whose rows stay in the cache."""
    tokens, seen, depth = [root], [1], [0]
    for branch in branches:
        mask = 1
        for i, t in enumerate(branch):
            mask |= 1 << len(tokens)
            tokens.append(t)
            seen.append(mask)
            depth.append(i + 1)
    start = model.cache.length(seq)
    words = torch.tensor(seen, dtype=torch.int64, device=model.device)
    logits = model.forward([seq], [tokens], positions=[start + d for d in depth], tree_mask=words)
    zeros = torch.zeros(len(tokens), device=model.device)
    best = sample(logits, zeros, temperature=zeros).tolist()
    keep, at = [0], 1
    for branch in branches:
        path, last = [0], 0
        for i, t in enumerate(branch):
            if best[last] != t:
                break
            last = at + i
            path.append(last)
        keep = max(keep, path, key=len)
        at += len(branch)
    model.cache.keep(seq, start, keep)
    return [tokens[i] for i in keep[1:]] + [best[keep[-1]]]


def main():
    model = Model(Config())
    prompt = torch.randint(0, model.c.vocab, (100,), generator=torch.Generator().manual_seed(1)).tolist()
    prompt += prompt[:30]  # something to look up
    seq, tokens, passes = decode(model, prompt, steps=40, n_drafts=5)
    print(f"{len(tokens) - len(prompt)} tokens in {passes} passes: {tokens[len(prompt):]}")

    model.cache.truncate(seq, len(tokens) - 1)
    twin = model.cache.fork(seq)  # shares every page until one of them writes
    logits = model.forward([seq, twin], [tokens[-1:], tokens[-1:]])
    u = torch.tensor([0.2, 0.8], device=model.device)
    first, second = sample(logits, u).tolist()
    print(f"two continuations of one prefix: {first}, {second}")

    accepted = verify_tree(model, seq, first, [[5, 6, 7], [8, 9]])
    print(f"tree: {len(accepted)} tokens, cache length {model.cache.length(seq)}")
    model.cache.free(twin)
    moved = model.cache.compact()
    print(f"compacted: {moved} pages moved, {model.cache.table.free_pages} of {model.c.pages} free")
    assert model.attention.status() == 0
    model.close()
    return tokens


if __name__ == "__main__":
    main()
