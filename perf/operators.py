"""The operators around the MoE layer in a decode/verify step, as cases that can be measured: norms and rotation of
queries and keys with the write into the paged cache, attention of new tokens over that cache, moving its pages, and
sampling from the logits.  `run` computes them in plain torch operations, or, with `own` set, through the package."""
import math
import random

import torch

own = False
DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # one verified chain of 6 drafted tokens at a middling context: the latency of a batch-1 step
        dict(name="attn_verify_chain", op="attn", dtype="bf16", batch=1, q_len=6, ctx=8192, ragged=False, heads=20,
             kv_heads=4, dim=128, page=64, tree=False, shape_seed=1),
        # a few sequences that each verify a tree of drafts; small heads, small pages
        dict(name="attn_verify_tree", op="attn", dtype="fp16", batch=4, q_len=24, ctx=4000, ragged=True, heads=16,
             kv_heads=2, dim=64, page=16, tree=True, shape_seed=2),
        # one token each of many sequences of very different lengths: the cache's bandwidth
        dict(name="attn_decode_batch", op="attn", dtype="bf16", batch=32, q_len=1, ctx=32768, ragged=True, heads=32,
             kv_heads=4, dim=128, page=16, tree=False, shape_seed=3),
        # the second half of a long prompt: the tensor cores
        dict(name="attn_prefill_chunk", op="attn", dtype="bf16", batch=1, q_len=8192, ctx=16384, ragged=False, heads=32,
             kv_heads=4, dim=128, page=64, tree=False, shape_seed=4),
        # chunks of several prompts at once, nothing a multiple of anything
        dict(name="attn_prefill_ragged", op="attn", dtype="fp16", batch=5, q_len=1501, ctx=6001, ragged=True, heads=14,
             kv_heads=2, dim=128, page=32, tree=False, shape_seed=5),
        # the same 6 tokens' queries, keys and values on their way into the cache: latency
        dict(name="rope_verify", op="rope", dtype="bf16", tokens=6, heads=20, kv_heads=4, dim=128, rot=128,
             interleaved=False, norm=True, page=64, far=8192),
        # partial rotation of interleaved pairs far into a long context
        dict(name="rope_partial_far", op="rope", dtype="fp16", tokens=1001, heads=16, kv_heads=2, dim=64, rot=32,
             interleaved=True, norm=True, page=16, far=1000000),
        # a prompt's chunk
        dict(name="rope_prefill", op="rope", dtype="bf16", tokens=16384, heads=32, kv_heads=4, dim=128, rot=128,
             interleaved=False, norm=True, page=64, far=32768),
        # a sequence is forked: its last, partly filled page is copied in every layer
        dict(name="pages_fork", op="pages", dtype="bf16", layers=42, pages=64, moves=1, kv_heads=4, dim=128, page=64),
        # a fragmented cache is compacted
        dict(name="pages_compact", op="pages", dtype="bf16", layers=8, pages=4096, moves=777, kv_heads=4, dim=128,
             page=16),
        # the verified positions' tokens from the model's vocabulary, every filter on
        dict(name="sample_verify", op="sample", rows=6, vocab=157184, params="nucleus"),
        # a full block of rows, each with settings of its own (greedy and unfiltered ones among them)
        dict(name="sample_mixed", op="sample", rows=64, vocab=157184, params="mixed"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "rope", "pages", "sample"])
    if op == "attn":
        while True:
            group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
            kv_heads = rng.choice([1, 2, 4, 8])
            kind = rng.choice(["decode", "verify", "tree", "prefill"])
            case = dict(op="attn", dtype=rng.choice(["bf16", "fp16"]),
                        batch=_log(rng, 1, 8 if kind == "prefill" else 48),
                        q_len={"decode": 1, "verify": _log(rng, 2, 64), "tree": _log(rng, 2, 64),
                               "prefill": _log(rng, 64, 8192)}[kind],
                        ctx=_log(rng, 100, 40000), ragged=rng.random() < 0.6, heads=group * kv_heads,
                        kv_heads=kv_heads, dim=rng.choice([64, 128, 128]), page=rng.choice([16, 32, 64, 128]),
                        tree=kind == "tree", shape_seed=rng.randrange(1 << 30))
            if case["ctx"] < case["q_len"] or case["heads"] > 64:
                continue
            w, most = work(case), work(listed()[3])
            # the plain form holds every score of the padded batch in 32 bits
            scores = case["batch"] * case["heads"] * case["q_len"] * case["ctx"]
            cache = case["batch"] * case["ctx"] * case["kv_heads"] * case["dim"]
            if w["flops"] <= most["flops"] and w["bytes"] <= 8e8 and scores <= 4.3e9 and cache <= 6e8:
                return case
    if op == "rope":
        dim = rng.choice([64, 128])
        kv_heads = rng.choice([1, 2, 4, 8])
        return dict(op="rope", dtype=rng.choice(["bf16", "fp16"]), tokens=_log(rng, 1, 12000),
                    heads=kv_heads * rng.choice([1, 3, 4, 5, 8]), kv_heads=kv_heads, dim=dim,
                    rot=rng.choice([dim, dim, dim // 2, dim // 4]), interleaved=rng.random() < 0.4,
                    norm=rng.random() < 0.8, page=rng.choice([16, 32, 64, 128]), far=_log(rng, 20000, 2000000))
    if op == "pages":
        pages = _log(rng, 4, 2048)
        return dict(op="pages", dtype=rng.choice(["bf16", "fp16"]), layers=rng.randint(1, 24), pages=pages,
                    moves=rng.randint(1, pages // 2), kv_heads=rng.choice([1, 2, 4]), dim=rng.choice([64, 128]),
                    page=rng.choice([16, 32, 64]))
    return dict(op="sample", rows=_log(rng, 1, 64), vocab=_log(rng, 100, 157184),
                params=rng.choice(["nucleus", "topk", "plain", "greedy", "mixed"]))


def _lens(case):
    """(new tokens, length with them) of each sequence of an attention case, from the case alone."""
    rng = random.Random(case["shape_seed"])
    q, kv = [], []
    for b in range(case["batch"]):
        qn, n = case["q_len"], case["ctx"]
        if case["ragged"] and b:  # the first sequence has the case's full lengths
            qn = qn if case["tree"] else rng.randint(max(1, qn // 4), qn)
            n = max(qn, _log(rng, max(1, n // 16), n))
        q.append(qn)
        kv.append(n)
    return q, kv


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype):
    return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)


def prepare(case, seed):
    return {"attn": _prepare_attn, "rope": _prepare_rope, "pages": _prepare_pages, "sample": _prepare_sample}[case["op"]](case, seed)


def run(state):
    return {"attn": _run_attn, "rope": _run_rope, "pages": _run_pages, "sample": _run_sample}[state["case"]["op"]](state)


def work(case):
    if case["op"] == "attn":
        q, kv = _lens(case)
        h, hk, d = case["heads"], case["kv_heads"], case["dim"]
        seen = sum(a * (n - a) + a * (a + 1) // 2 for a, n in zip(q, kv))
        return {"bytes": 2 * d * (2 * hk * sum(kv) + 2 * h * sum(q)) + 4 * h * sum(q), "flops": 4 * h * d * seen}
    if case["op"] == "rope":
        n = case["tokens"] * (case["heads"] + 2 * case["kv_heads"]) * case["dim"]
        return {"bytes": 4 * n, "flops": 8 * n}
    if case["op"] == "pages":
        n = case["layers"] * case["moves"] * case["page"] * case["kv_heads"] * case["dim"]
        return {"bytes": 8 * n, "flops": 0}
    return {"bytes": 4 * case["rows"] * case["vocab"], "flops": 8 * case["rows"] * case["vocab"]}


# ---- attention of new tokens over the paged cache ---------------------------------------------------------------------


def _prepare_attn(case, seed):
    g, dt = _gen(seed), DTYPES[case["dtype"]]
    q_lens, kv_lens = _lens(case)
    page, d, hk = case["page"], case["dim"], case["kv_heads"]
    need = [-(-n // page) for n in kv_lens]
    width, total = max(need), sum(need) + 3
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    table = torch.full((case["batch"], width), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    starts = [0]
    for n in q_lens:
        starts.append(starts[-1] + n)
    state = dict(case=case, q=_randn(g, starts[-1], case["heads"], d, dtype=dt),
                 k_cache=_randn(g, total, page, hk, d, dtype=dt), v_cache=_randn(g, total, page, hk, d, dtype=dt),
                 table=table, starts=torch.tensor(starts, dtype=torch.int32, device=DEV),
                 kv_lens=torch.tensor(kv_lens, dtype=torch.int32, device=DEV), max_q=max(q_lens), max_kv=max(kv_lens),
                 scale=d ** -0.5, tree=None)
    if case["tree"]:
        # token i of a tree sees itself and its ancestors: a bit for each of the chunk's tokens
        n, rows = case["q_len"], []
        rng = random.Random(seed)
        for _ in range(case["batch"]):
            seen = []
            for i in range(n):
                parent = rng.randrange(-1, i) if i else -1
                seen.append((seen[parent] if parent >= 0 else 0) | (1 << i))
            rows += [s - (1 << 64) if s >> 63 else s for s in seen]
        state["tree"] = torch.tensor(rows, dtype=torch.int64, device=DEV)
    if own:
        from weight_streaming_expert_gb300 import PagedAttention
        state["attn"] = PagedAttention(case["heads"], hk, d)
    return state


def _run_attn(s):
    if own:
        return s["attn"](s["q"], s["k_cache"], s["v_cache"], s["table"], s["starts"], s["kv_lens"], s["max_q"],
                         scale=s["scale"], tree_mask=s["tree"], return_lse=True)
    # the batch padded to its longest sequence and chunk
    c, q = s["case"], s["q"]
    group, page = c["heads"] // c["kv_heads"], c["page"]
    starts, kv_lens = s["starts"].long(), s["kv_lens"].long()
    q_lens = starts[1:] - starts[:-1]
    pos = torch.arange(s["max_kv"], device=DEV)
    tok = torch.arange(s["max_q"], device=DEV)
    held = pos[None, :] < kv_lens[:, None]
    slots = s["table"].long().clamp_min(0)[:, pos // page] * page + pos % page
    k = s["k_cache"].flatten(0, 1)[slots].float()  # [B, n, Hk, D]
    v = s["v_cache"].flatten(0, 1)[slots].float().masked_fill(~held[:, :, None, None], 0.0)
    rows = (starts[:-1, None] + tok[None, :]).clamp_max(q.shape[0] - 1)
    qp = q[rows].float().unflatten(2, (c["kv_heads"], group))  # [B, m, Hk, G, D]
    qp = qp.permute(0, 2, 3, 1, 4).flatten(2, 3)  # [B, Hk, G m, D]
    scores = torch.matmul(qp, k.permute(0, 2, 3, 1)).mul_(s["scale"]).unflatten(2, (group, s["max_q"]))
    own_at = (kv_lens - q_lens)[:, None] + tok[None, :]  # each token's place in its sequence
    sees = (pos[None, None, :] <= own_at[:, :, None]) & held[:, None, :]
    if s["tree"] is not None:
        bit = pos[None, None, :] - (kv_lens - q_lens)[:, None, None]
        inside = bit >= 0
        sees = held[:, None, :] & (~inside | ((s["tree"][rows][:, :, None] >> bit.clamp(0, 63)) & 1).bool())
    scores.masked_fill_(~sees[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = scores.sub_(top).exp_()
    total = p.sum(-1)
    out = torch.matmul(p.flatten(2, 3), v.permute(0, 2, 1, 3)).unflatten(2, (group, s["max_q"]))
    out = out / torch.where(total == 0, torch.ones_like(total), total)[..., None]
    lse = total.log() + top[..., 0]
    mine = (tok[None, :] < q_lens[:, None])
    out = out.permute(0, 3, 1, 2, 4).flatten(2, 3)[mine].to(q.dtype)  # [T, H, D]
    lse = lse.permute(0, 3, 1, 2).flatten(2, 3)[mine].contiguous()
    return out, lse


def _exact_attn(s):
    c = s["case"]
    q_lens, kv_lens = _lens(c)
    group, page = c["heads"] // c["kv_heads"], c["page"]
    outs, lses, at = [], [], 0
    for b, (m, n) in enumerate(zip(q_lens, kv_lens)):
        pages = s["table"][b, :-(-n // page)].long()
        heads_o, heads_l = [], []
        i = torch.arange(m, device=DEV)[:, None]
        j = torch.arange(n, device=DEV)[None, :]
        hidden = j > n - m + i
        if s["tree"] is not None:
            bits = s["tree"][at:at + m][:, None]
            hidden = (j >= n - m) & (((bits >> (j - (n - m)).clamp(min=0)) & 1) == 0)
        for h in range(c["heads"]):
            k = s["k_cache"][pages, :, h // group].reshape(-1, c["dim"])[:n].double()
            v = s["v_cache"][pages, :, h // group].reshape(-1, c["dim"])[:n].double()
            x = (s["q"][at:at + m, h].double() @ k.T) * s["scale"]
            x[hidden] = -math.inf
            lse = torch.logsumexp(x, 1)
            heads_l.append(lse)
            heads_o.append(torch.exp(x - lse[:, None]) @ v)
        outs.append(torch.stack(heads_o, 1))
        lses.append(torch.stack(heads_l, 1))
        at += m
    return torch.cat(outs), torch.cat(lses)


# ---- norms and rotation of queries and keys, into the cache -----------------------------------------------------------


def _prepare_rope(case, seed):
    g, dt = _gen(seed), DTYPES[case["dtype"]]
    t, h, hk, d, page = case["tokens"], case["heads"], case["kv_heads"], case["dim"], case["page"]
    pages = -(-t // page) + 2
    qkv = _randn(g, t, h + 2 * hk, d, dtype=dt) * 1.5  # one projection's output
    first = int(torch.randint(0, max(1, case["far"] - t), (1,), generator=g, device=DEV))
    # the tokens follow one another in a sequence whose pages lie anywhere
    order = torch.randperm(pages, generator=g, device=DEV)
    at = torch.arange(t, device=DEV) + first % page
    state = dict(case=case, q=qkv[:, :h], k=qkv[:, h:h + hk], v=qkv[:, h + hk:],
                 q_weight=None, k_weight=None, positions=torch.arange(first, first + t, device=DEV, dtype=torch.int32),
                 slots=order[at // page] * page + at % page, theta=1e6, eps=1e-6,
                 k_cache=_randn(g, pages, page, hk, d, dtype=dt), v_cache=_randn(g, pages, page, hk, d, dtype=dt))
    if case["norm"]:
        state["q_weight"] = (1 + 0.2 * _randn(g, d, dtype=torch.float32)).to(dt)
        state["k_weight"] = (1 + 0.2 * _randn(g, d, dtype=torch.float32)).to(dt)
    if own:
        from weight_streaming_expert_gb300 import QKNormRope
        state["op"] = QKNormRope(d, rotary_dim=case["rot"], theta=state["theta"], interleaved=case["interleaved"],
                                 eps=state["eps"])
    return state


def _run_rope(s):
    if own:
        q = s["op"](s["q"], s["k"], s["v"], s["q_weight"], s["k_weight"], s["positions"], s["slots"], s["k_cache"],
                    s["v_cache"])
        return q, s["k_cache"], s["v_cache"]
    c = s["case"]
    rot = c["rot"]
    # angles of far positions need 64 bits
    freq = s["theta"] ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    angle = s["positions"].double()[:, None] * freq
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turned(x, w):
        x = x.float()
        if w is not None:
            x = x * (x.square().mean(-1, keepdim=True) + s["eps"]).rsqrt() * w.float()
        r, rest = x[..., :rot], x[..., rot:]
        if c["interleaved"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
        else:
            a, b = r[..., :rot // 2], r[..., rot // 2:]
            r = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
        return torch.cat((r, rest), -1).to(s["q"].dtype)

    s["k_cache"].flatten(0, 1)[s["slots"]] = turned(s["k"], s["k_weight"])
    s["v_cache"].flatten(0, 1)[s["slots"]] = s["v"]
    return turned(s["q"], s["q_weight"]), s["k_cache"], s["v_cache"]


def _exact_rope(s):
    c = s["case"]
    rot, d = c["rot"], c["dim"]
    n = torch.arange(rot // 2, device=DEV, dtype=torch.float64)
    angle = s["positions"].double()[:, None] * torch.exp(-(2 * n / rot) * math.log(s["theta"]))
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]
    first = torch.arange(0, rot, 2, device=DEV) if c["interleaved"] else torch.arange(rot // 2, device=DEV)
    second = first + (1 if c["interleaved"] else rot // 2)

    def turned(x, w):
        y = x.double()
        if w is not None:
            y = y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / d + s["eps"]) * w.double()
        z = torch.complex(y[..., first], y[..., second]) * turn
        y = y.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    page, off = s["slots"] // c["page"], s["slots"] % c["page"]
    k_cache[page, off] = turned(s["k"], s["k_weight"])
    v_cache[page, off] = s["v"].double()
    return turned(s["q"], s["q_weight"]), k_cache, v_cache


# ---- pages of the cache -----------------------------------------------------------------------------------------------


def _prepare_pages(case, seed):
    g, dt = _gen(seed), DTYPES[case["dtype"]]
    shape = (case["layers"], case["pages"], case["page"], case["kv_heads"], case["dim"])
    order = torch.randperm(case["pages"], generator=g, device=DEV).to(torch.int32)
    return dict(case=case, k_pool=_randn(g, *shape, dtype=dt), v_pool=_randn(g, *shape, dtype=dt),
                src=order[:case["moves"]].contiguous(), dst=order[case["moves"]:2 * case["moves"]].contiguous())


def _run_pages(s):
    if own:
        from weight_streaming_expert_gb300 import copy_pages
        copy_pages(s["k_pool"], s["v_pool"], s["src"], s["dst"])
    else:
        src, dst = s["src"].long(), s["dst"].long()
        s["k_pool"][:, dst] = s["k_pool"][:, src]
        s["v_pool"][:, dst] = s["v_pool"][:, src]
    return s["k_pool"], s["v_pool"]


def _exact_pages(s):
    out = []
    for pool in (s["k_pool"], s["v_pool"]):
        moved = pool.clone()
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            moved[:, b] = pool[:, a]
        out.append(moved)
    return tuple(out)


# ---- sampling ---------------------------------------------------------------------------------------------------------

#: A token's weight is exp((logit - largest) / temperature) in 32 bits, held as a whole number of 2^-38: sums of whole
#: numbers have one value whatever their order, so the token does not depend on who adds them up.
ONE = 1 << 38


def _prepare_sample(case, seed):
    g, m, v = _gen(seed), case["rows"], case["vocab"]
    # logits of a trained model: a broad bulk and a few that stand out
    logits = _randn(g, m, v, dtype=torch.float32) * 2.0
    logits += 7.0 * torch.rand(m, v, generator=g, device=DEV).pow(12)
    kinds = {"nucleus": [(0.8, 50, 0.95, 0.02)], "topk": [(1.0, 40, 1.0, 0.0)], "plain": [(1.0, 0, 1.0, 0.0)],
             "greedy": [(0.0, 0, 1.0, 0.0)],
             "mixed": [(0.7, 0, 0.9, 0.0), (0.0, 0, 1.0, 0.0), (1.0, 0, 1.0, 0.0), (1.3, 1000, 0.99, 0.0),
                       (1.0, 0, 1.0, 0.05), (0.6, 20, 1.0, 0.0), (0.9, 0, 0.5, 0.1)]}[case["params"]]
    rows = [kinds[i % len(kinds)] for i in range(m)]
    column = lambda i, dt: torch.tensor([r[i] for r in rows], dtype=dt, device=DEV)
    return dict(case=case, logits=logits, u=torch.rand(m, generator=g, device=DEV), temperature=column(0, torch.float32),
                top_k=column(1, torch.int32), top_p=column(2, torch.float32), min_p=column(3, torch.float32))


def _run_sample(s):
    if own:
        from weight_streaming_expert_gb300 import sample
        return sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                      min_p=s["min_p"], return_probs=True)
    x, v = s["logits"], s["logits"].shape[1]
    best, order = x.sort(dim=1, descending=True, stable=True)
    t = s["temperature"][:, None]
    greedy = t <= 0
    e = ((best - best[:, :1]) / torch.where(greedy, torch.ones_like(t), t)).exp()
    weight = (e * ONE).long()
    rank = torch.arange(v, device=DEV)[None, :]
    k = torch.where(greedy, torch.ones_like(s["top_k"][:, None]), s["top_k"][:, None])
    keep = (k <= 0) | (rank < k)
    weight = torch.where(keep, weight, 0)
    before = weight.cumsum(1) - weight
    p = s["top_p"][:, None].double()
    keep &= (p >= 1) | (rank == 0) | (before.double() < p * weight.sum(1, keepdim=True).double())
    keep &= weight.double() >= s["min_p"][:, None].double() * ONE
    weight = torch.where(keep, weight, 0)
    total = weight.sum(1, keepdim=True)
    by_token = torch.zeros_like(weight).scatter_(1, order, weight)
    wanted = (s["u"][:, None].double() * total.double()).long()
    token = (by_token.cumsum(1) <= wanted).sum(1, keepdim=True)
    prob = by_token.gather(1, token).double() / total.double()
    return token[:, 0].to(torch.int32), prob[:, 0].float()


def _exact_sample(s):
    """None where a row's outcome hangs on less than 32 bits can tell: a filter's border, or the drawn token's."""
    close, tokens, probs = 1e-7, [], []
    for i in range(s["case"]["rows"]):
        x = s["logits"][i].double()
        t, k, p, least = (float(s[n][i]) for n in ("temperature", "top_k", "top_p", "min_p"))
        values, order = torch.sort(x, descending=True, stable=True)
        if t <= 0:
            tokens.append(int(order[0]))
            probs.append(1.0)
            continue
        w = torch.exp((values - values[0]) / t)
        n = min(int(k), len(w)) if k > 0 else len(w)
        w, order = w[:n], order[:n]
        if p < 1:
            cum = torch.cumsum(w, 0) / w.sum()
            n = int((cum < p).sum()) + 1
            if float((cum - p).abs().min()) < close:
                return None
            w, order = w[:n], order[:n]
        if least > 0:
            if float((w / least - 1).abs().min()) < 20 * close:
                return None
            w, order = w[w >= least], order[:int((w >= least).sum())]
        order, back = torch.sort(order)
        cum = torch.cumsum(w[back], 0) / w.sum()
        u = float(s["u"][i])
        if len(cum) > 1 and float((cum[:-1] - u).abs().min()) < close:
            return None
        at = min(int((cum <= u).sum()), len(cum) - 1)
        tokens.append(int(order[at]))
        probs.append(float(w[back][at] / w.sum()))
    return torch.tensor(tokens, dtype=torch.int32), torch.tensor(probs, dtype=torch.float64)


def exact(case, seed):
    state = prepare(case, seed)
    return {"attn": _exact_attn, "rope": _exact_rope, "pages": _exact_pages, "sample": _exact_sample}[case["op"]](state)
