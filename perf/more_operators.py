"""What a served batch adds to a decode/verify step, as cases that can be measured: keys and values quantised to E4M3 as
they enter the paged cache and read back, attention over that cache, attention of a batch whose sequences begin with the
same pages, and penalties, biases and grammar masks on the logits.  `run` computes them in plain torch operations, or,
with `own` set, through the package."""
import math
import random

import torch

own = False
DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # the verified chain of a batch-1 step on its way into the cache, and back: latency
        dict(name="kv8_verify", op="kv8", dtype="bf16", tokens=6, heads=20, kv_heads=4, dim=128, rot=128,
             interleaved=False, norm=True, page=64, far=8192),
        # small heads, pairs side by side, only part of a head turned, an odd number of tokens
        dict(name="kv8_partial", op="kv8", dtype="fp16", tokens=1001, heads=16, kv_heads=2, dim=64, rot=32,
             interleaved=True, norm=True, page=16, far=1000000),
        # a prompt's chunk
        dict(name="kv8_prompt", op="kv8", dtype="bf16", tokens=16384, heads=32, kv_heads=4, dim=128, rot=128,
             interleaved=False, norm=True, page=64, far=32768),
        # one verified chain at a middling context: latency
        dict(name="attn8_verify", op="attn", quant=True, dtype="bf16", batch=1, q_len=6, prefix=0, ctx=8192,
             ragged=False, heads=20, kv_heads=4, dim=128, page=64, tree=False, shape_seed=1),
        # one token each of many sequences of very different lengths: the cache's bandwidth
        dict(name="attn8_decode_batch", op="attn", quant=True, dtype="bf16", batch=32, q_len=1, prefix=0, ctx=32768,
             ragged=True, heads=32, kv_heads=4, dim=128, page=16, tree=False, shape_seed=3),
        # chunks of several prompts at once, nothing a multiple of anything
        dict(name="attn8_prefill_ragged", op="attn", quant=True, dtype="fp16", batch=5, q_len=1501, prefix=0, ctx=6001,
             ragged=True, heads=14, kv_heads=2, dim=128, page=32, tree=False, shape_seed=5),
        # several answers drawn for one prompt
        dict(name="prefix_samples", op="attn", quant=False, dtype="bf16", batch=8, q_len=1, prefix=8192, ctx=300,
             ragged=True, heads=20, kv_heads=4, dim=128, page=64, tree=False, shape_seed=6),
        # trees of drafts after a common instruction, small heads, an E4M3 cache
        dict(name="prefix8_verify_trees", op="attn", quant=True, dtype="fp16", batch=12, q_len=13, prefix=4000,
             ctx=700, ragged=True, heads=16, kv_heads=2, dim=64, page=16, tree=True, shape_seed=7),
        # a large batch behind a long common document
        dict(name="prefix_batch", op="attn", quant=False, dtype="bf16", batch=128, q_len=1, prefix=16384, ctx=2000,
             ragged=True, heads=32, kv_heads=4, dim=128, page=64, tree=False, shape_seed=8),
        # the verified positions of one sequence, whose histories grow by one token from row to row: latency
        dict(name="logits_verify", op="logits", rows=6, vocab=157184, history=4000, chain=True, biases=20, mask=True),
        # a vocabulary that is a multiple of nothing, no grammar
        dict(name="logits_odd", op="logits", rows=33, vocab=32001, history=700, chain=False, biases=100, mask=False),
        # a batch of sequences, each with a history and a grammar of its own
        dict(name="logits_batch", op="logits", rows=64, vocab=157184, history=8000, chain=False, biases=300, mask=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["kv8", "attn", "attn", "attn", "logits"])
    if op == "attn":
        most = [work(c) for c in listed() if c["op"] == "attn"]
        while True:
            shared = rng.random() < 0.5
            group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
            kv_heads = rng.choice([1, 2, 4, 8])
            page = rng.choice([16, 32, 64, 128])
            kind = rng.choice(["decode", "decode", "verify", "tree", "prefill"])
            case = dict(op="attn", quant=not shared or rng.random() < 0.4, dtype=rng.choice(["bf16", "fp16"]),
                        batch=_log(rng, 2 if shared else 1, 8 if kind == "prefill" else 128 if shared else 48),
                        q_len={"decode": 1, "verify": _log(rng, 2, 64), "tree": _log(rng, 2, 64),
                               "prefill": _log(rng, 64, 2048)}[kind],
                        prefix=_log(rng, 200, 32000) // page * page if shared else 0, ctx=_log(rng, 30, 40000),
                        ragged=rng.random() < 0.7, heads=group * kv_heads, kv_heads=kv_heads,
                        dim=rng.choice([64, 128, 128]), page=page, tree=kind == "tree",
                        shape_seed=rng.randrange(1 << 30))
            if case["ctx"] < case["q_len"] or case["heads"] > 64:
                continue
            w = work(case)
            # the plain form holds every score of the padded batch in 32 bits
            scores = case["batch"] * case["heads"] * case["q_len"] * (case["prefix"] + case["ctx"])
            cache = (case["batch"] * case["ctx"] + case["prefix"]) * case["kv_heads"] * case["dim"]
            if (w["flops"] <= max(m["flops"] for m in most) and w["bytes"] <= max(m["bytes"] for m in most)
                    and scores <= 2.5e9 and cache <= 6e8):
                return case
    if op == "kv8":
        dim = rng.choice([64, 128])
        kv_heads = rng.choice([1, 2, 4, 8])
        return dict(op="kv8", dtype=rng.choice(["bf16", "fp16"]), tokens=_log(rng, 1, 12000),
                    heads=kv_heads * rng.choice([1, 3, 4, 5]), kv_heads=kv_heads, dim=dim,
                    rot=rng.choice([dim, dim, dim // 2, dim // 4]), interleaved=rng.random() < 0.4,
                    norm=rng.random() < 0.8, page=rng.choice([16, 32, 64, 128]), far=_log(rng, 20000, 2000000))
    return dict(op="logits", rows=_log(rng, 1, 64), vocab=_log(rng, 100, 157184), history=_log(rng, 1, 8000),
                chain=rng.random() < 0.4, biases=rng.choice([0, 1, 30, 300]), mask=rng.random() < 0.6)


def _lens(case):
    """(new tokens, positions after the prefix with them) of each sequence of an attention case, from the case alone."""
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
    return {"kv8": _prepare_kv8, "attn": _prepare_attn, "logits": _prepare_logits}[case["op"]](case, seed)


def run(state):
    return {"kv8": _run_kv8, "attn": _run_attn, "logits": _run_logits}[state["case"]["op"]](state)


def work(case):
    if case["op"] == "attn":
        q, kv = _lens(case)
        h, hk, d = case["heads"], case["kv_heads"], case["dim"]
        seen = sum(a * (case["prefix"] + n - a) + a * (a + 1) // 2 for a, n in zip(q, kv))
        row = d + 1 if case["quant"] else 2 * d
        return {"bytes": 2 * hk * row * (case["prefix"] + sum(kv)) + 4 * d * h * sum(q) + 4 * h * sum(q),
                "flops": 4 * h * d * seen}
    if case["op"] == "kv8":
        t, h, hk, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
        return {"bytes": t * (4 * h * d + 4 * hk * d + 4 * hk * (d + 1) + 4 * hk * d), "flops": 10 * t * (h + 2 * hk) * d}
    n = case["rows"] * case["vocab"]
    return {"bytes": 8 * n + (n // 8 if case["mask"] else 0) + 4 * case["rows"] * case["history"] // (case["rows"] if case["chain"] else 1),
            "flops": 4 * n}


# ---- E4M3 with a power of two for each row ----------------------------------------------------------------------------


def _quantise(x):
    """fp32 [..., D] to codes and the exponent of each row: the least with |x| <= 448 * 2^e, in -40..40."""
    mantissa, e = torch.frexp(x.abs().amax(-1))
    e = (e - torch.where(mantissa <= 0.875, 9, 8)).clamp(-40, 40)
    scaled = torch.ldexp(x, -e[..., None]).clamp(-448.0, 448.0)
    return scaled.to(torch.float8_e4m3fn), e


def _values(codes, scale):
    """What codes [..., D] with scale bytes [...] stand for, in fp32."""
    return codes.float() * torch.exp2(scale.float() - 127.0)[..., None]


def _rows_of(codes, scale, slots):
    """Codes [pages, page, Hk, D] and scales [pages, Hk, page] of slots, as values."""
    picked = codes.view(torch.uint8).flatten(0, 1)[slots].view(torch.float8_e4m3fn)
    return _values(picked, scale.transpose(1, 2).flatten(0, 1)[slots])


# ---- keys and values into the E4M3 cache, and back --------------------------------------------------------------------


def _prepare_kv8(case, seed):
    g, dt = _gen(seed), DTYPES[case["dtype"]]
    t, h, hk, d, page = case["tokens"], case["heads"], case["kv_heads"], case["dim"], case["page"]
    pages = -(-t // page) + 2
    qkv = _randn(g, t, h + 2 * hk, d, dtype=dt) * 1.5  # one projection's output
    qkv[:, h + hk:] *= torch.exp2(4.0 * torch.rand(t, hk, 1, generator=g, device=DEV) - 3.0).to(dt)
    first = int(torch.randint(0, max(1, case["far"] - t), (1,), generator=g, device=DEV))
    # the tokens follow one another in a sequence whose pages lie anywhere
    order = torch.randperm(pages, generator=g, device=DEV)
    at = torch.arange(t, device=DEV) + first % page
    empty = lambda *shape: torch.zeros(*shape, dtype=torch.uint8, device=DEV)
    state = dict(case=case, q=qkv[:, :h], k=qkv[:, h:h + hk], v=qkv[:, h + hk:], q_weight=None, k_weight=None,
                 positions=torch.arange(first, first + t, device=DEV, dtype=torch.int32),
                 slots=order[at // page] * page + at % page, theta=1e6, eps=1e-6,
                 k_cache=empty(pages, page, hk, d).view(torch.float8_e4m3fn),
                 v_cache=empty(pages, page, hk, d).view(torch.float8_e4m3fn),
                 k_scale=empty(pages, hk, page), v_scale=empty(pages, hk, page))
    if case["norm"]:
        state["q_weight"] = (1 + 0.2 * _randn(g, d, dtype=torch.float32)).to(dt)
        state["k_weight"] = (1 + 0.2 * _randn(g, d, dtype=torch.float32)).to(dt)
    if own:
        from weight_streaming_expert_gb300 import QKNormRope
        state["op"] = QKNormRope(d, rotary_dim=case["rot"], theta=state["theta"], interleaved=case["interleaved"],
                                 eps=state["eps"])
    return state


def _run_kv8(s):
    dt = s["q"].dtype
    if own:
        from weight_streaming_expert_gb300 import read_cache
        q = s["op"](s["q"], s["k"], s["v"], s["q_weight"], s["k_weight"], s["positions"], s["slots"], s["k_cache"],
                    s["v_cache"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        return (q,) + tuple(read_cache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["slots"], dtype=dt))
    c = s["case"]
    rot, page = c["rot"], c["page"]
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
        return torch.cat((r, rest), -1)

    pg, row = s["slots"] // page, s["slots"] % page
    codes, e = _quantise(turned(s["k"], s["k_weight"]))
    s["k_cache"].view(torch.uint8)[pg, row] = codes.view(torch.uint8)
    s["k_scale"].transpose(1, 2)[pg, row] = (e + 127).to(torch.uint8)
    codes, e = _quantise(s["v"].float())
    s["v_cache"].view(torch.uint8)[pg, row] = codes.view(torch.uint8)
    s["v_scale"].transpose(1, 2)[pg, row] = (e + 127).to(torch.uint8)
    return (turned(s["q"], s["q_weight"]).to(dt), _rows_of(s["k_cache"], s["k_scale"], s["slots"]).to(dt),
            _rows_of(s["v_cache"], s["v_scale"], s["slots"]).to(dt))


def _exact_kv8(s):
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

    def held(y):
        # four significant bits, steps of at least 2^-9, around a power of two that takes the largest to at most 448
        largest = y.abs().max(-1, keepdim=True).values
        scale = torch.exp2(torch.ceil(torch.log2(largest.clamp_min(2.0 ** -60) / 448)).clamp(-40, 40))
        x = y / scale
        step = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))) - 3)
        return (torch.round(x / step) * step).clamp(-448, 448) * scale

    return turned(s["q"], s["q_weight"]), held(turned(s["k"], s["k_weight"])), held(s["v"].double())


# ---- attention of new tokens over the paged cache ---------------------------------------------------------------------


def _prepare_attn(case, seed):
    g, dt = _gen(seed), DTYPES[case["dtype"]]
    q_lens, own_lens = _lens(case)
    page, d, hk = case["page"], case["dim"], case["kv_heads"]
    shared = case["prefix"] // page
    need = [-(-n // page) for n in own_lens]
    width, total = shared + max(need), shared + sum(need) + 3
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    table = torch.full((case["batch"], width), -1, dtype=torch.int32, device=DEV)
    table[:, :shared] = order[:shared]
    at = shared
    for b, n in enumerate(need):
        table[b, shared:shared + n] = order[at:at + n]
        at += n
    starts = [0]
    for n in q_lens:
        starts.append(starts[-1] + n)
    state = dict(case=case, q=_randn(g, starts[-1], case["heads"], d, dtype=dt),
                 k_cache=_randn(g, total, page, hk, d, dtype=dt), v_cache=_randn(g, total, page, hk, d, dtype=dt),
                 k_scale=None, v_scale=None, table=table, starts=torch.tensor(starts, dtype=torch.int32, device=DEV),
                 kv_lens=torch.tensor([case["prefix"] + n for n in own_lens], dtype=torch.int32, device=DEV),
                 max_q=max(q_lens), max_own=max(own_lens), scale=d ** -0.5, tree=None)
    if case["quant"]:
        for name in ("k", "v"):
            codes, e = _quantise(state[name + "_cache"].float())
            state[name + "_cache"] = codes
            state[name + "_scale"] = (e + 127).to(torch.uint8).transpose(1, 2).contiguous()
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


def _rows(s, cache, scale, slots):
    return cache.flatten(0, 1)[slots].float() if scale is None else _rows_of(cache, scale, slots)


def _run_attn(s):
    c, q = s["case"], s["q"]
    if own:
        return s["attn"](q, s["k_cache"], s["v_cache"], s["table"], s["starts"], s["kv_lens"], s["max_q"],
                         scale=s["scale"], tree_mask=s["tree"], return_lse=True, k_scale=s["k_scale"],
                         v_scale=s["v_scale"], prefix_len=c["prefix"])
    # every token against the prefix, and the batch padded to its longest sequence and chunk against the rest
    group, page, m, hk = c["heads"] // c["kv_heads"], c["page"], s["max_q"], c["kv_heads"]
    shared = c["prefix"] // page
    starts, lens = s["starts"].long(), s["kv_lens"].long() - c["prefix"]
    q_lens = starts[1:] - starts[:-1]
    pos, tok = torch.arange(s["max_own"], device=DEV), torch.arange(m, device=DEV)
    held = pos[None, :] < lens[:, None]
    slots = s["table"].long().clamp_min(0)[:, shared + pos // page] * page + pos % page
    k = _rows(s, s["k_cache"], s["k_scale"], slots)  # [B, n, Hk, D]
    v = _rows(s, s["v_cache"], s["v_scale"], slots).masked_fill(~held[:, :, None, None], 0.0)
    rows = (starts[:-1, None] + tok[None, :]).clamp_max(q.shape[0] - 1)
    qp = q[rows].float().unflatten(2, (hk, group))  # [B, m, Hk, G, D]
    qp = qp.permute(0, 2, 3, 1, 4).flatten(2, 3)  # [B, Hk, G m, D]
    scores = torch.matmul(qp, k.permute(0, 2, 3, 1)).mul_(s["scale"]).unflatten(2, (group, m))
    own_at = (lens - q_lens)[:, None] + tok[None, :]  # each token's place after the prefix
    sees = (pos[None, None, :] <= own_at[:, :, None]) & held[:, None, :]
    if s["tree"] is not None:
        bit = pos[None, None, :] - (lens - q_lens)[:, None, None]
        sees = held[:, None, :] & ((bit < 0) | ((s["tree"][rows][:, :, None] >> bit.clamp(0, 63)) & 1).bool())
    scores.masked_fill_(~sees[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    if shared:
        before = torch.arange(c["prefix"], device=DEV)
        slots = s["table"].long()[0, before // page] * page + before % page
        k0 = _rows(s, s["k_cache"], s["k_scale"], slots)  # [P, Hk, D]
        v0 = _rows(s, s["v_cache"], s["v_scale"], slots)
        far = torch.matmul(qp, k0.permute(1, 2, 0)).mul_(s["scale"]).unflatten(2, (group, m))
        top = torch.maximum(top, far.amax(-1, keepdim=True))
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = scores.sub_(top).exp_()
    total = p.sum(-1)
    out = torch.matmul(p.flatten(2, 3), v.permute(0, 2, 1, 3)).unflatten(2, (group, m))
    if shared:
        p = far.sub_(top).exp_()
        total = total + p.sum(-1)
        out = out + torch.matmul(p.flatten(2, 3), v0.permute(1, 0, 2)).unflatten(2, (group, m))
    out = out / torch.where(total == 0, torch.ones_like(total), total)[..., None]
    lse = total.log() + top[..., 0]
    mine = tok[None, :] < q_lens[:, None]
    out = out.permute(0, 3, 1, 2, 4).flatten(2, 3)[mine].to(q.dtype)  # [T, H, D]
    return out, lse.permute(0, 3, 1, 2).flatten(2, 3)[mine].contiguous()


def _exact_attn(s):
    c = s["case"]
    q_lens, own_lens = _lens(c)
    group, page = c["heads"] // c["kv_heads"], c["page"]

    def values(cache, scale, pages, head, n):
        x = cache[pages, :, head] if scale is None else cache.view(torch.uint8)[pages, :, head].view(torch.float8_e4m3fn)
        x = x.double()
        if scale is not None:
            x = x * torch.pow(2.0, scale[pages, head].double() - 127)[..., None]
        return x.reshape(-1, c["dim"])[:n]

    outs, lses, at = [], [], 0
    for b, (m, n) in enumerate(zip(q_lens, own_lens)):
        n += c["prefix"]
        pages = s["table"][b, :-(-n // page)].long()
        heads_o, heads_l = [], []
        i = torch.arange(m, device=DEV)[:, None]
        j = torch.arange(n, device=DEV)[None, :]
        hidden = j > n - m + i
        if s["tree"] is not None:
            bits = s["tree"][at:at + m][:, None]
            hidden = (j >= n - m) & (((bits >> (j - (n - m)).clamp(min=0)) & 1) == 0)
        for hk in range(c["kv_heads"]):
            k, v = values(s["k_cache"], s["k_scale"], pages, hk, n), values(s["v_cache"], s["v_scale"], pages, hk, n)
            x = torch.matmul(s["q"][at:at + m, hk * group:(hk + 1) * group].double().transpose(0, 1), k.T) * s["scale"]
            x = x.masked_fill(hidden, -math.inf)
            lse = torch.logsumexp(x, -1)
            heads_l.append(lse)
            heads_o.append(torch.exp(x - lse[..., None]) @ v)
        outs.append(torch.cat(heads_o).transpose(0, 1))
        lses.append(torch.cat(heads_l).transpose(0, 1))
        at += m
    return torch.cat(outs), torch.cat(lses)


# ---- penalties, biases and grammar masks ------------------------------------------------------------------------------


def _prepare_logits(case, seed):
    g, m, vocab, n = _gen(seed), case["rows"], case["vocab"], case["history"]
    rand = lambda *shape: torch.rand(*shape, generator=g, device=DEV)
    logits = _randn(g, m, vocab, dtype=torch.float32) * 2.0
    logits += 7.0 * rand(m, vocab).pow(12)
    # text repeats itself: few tokens make up most of it
    tokens = lambda k: (rand(k).pow(4) * vocab).long().clamp_max(vocab - 1).to(torch.int32)
    if case["chain"]:  # row i: the sequence up to its i-th draft
        begin, end = torch.zeros(m, device=DEV), n + torch.arange(m, device=DEV)
        answer = torch.full((m,), n // 2, device=DEV)
        history = tokens(n + m)
    else:
        lens = 1 + (n * rand(m)).long()
        lens[0] = n
        end = lens.cumsum(0)
        begin = end - lens
        answer = begin + (lens * rand(m)).long()
        history = tokens(int(end[-1]))
    counts = (case["biases"] * rand(m)).long()
    counts[0] = case["biases"]
    starts = torch.cat((torch.zeros(1, dtype=torch.long, device=DEV), counts.cumsum(0)))
    state = dict(case=case, logits=logits, history=history, spans=torch.stack((begin, answer, end), 1).to(torch.int32),
                 repetition=1.0 + 0.4 * rand(m), presence=0.6 * rand(m), frequency=0.3 * rand(m), bias_ids=None,
                 bias_values=None, bias_starts=None, allowed=None)
    if case["biases"]:
        state.update(bias_ids=tokens(int(starts[-1])), bias_values=_randn(g, int(starts[-1]), dtype=torch.float32) * 3.0,
                     bias_starts=starts.to(torch.int32))
    if case["mask"]:
        # a grammar leaves most tokens, some, or few
        words = lambda: torch.randint(0, 1 << 32, (m, -(-vocab // 32)), generator=g, device=DEV)
        kind = torch.arange(m, device=DEV)[:, None] % 3
        bits = torch.where(kind == 0, words() | words() | words(), torch.where(kind == 1, words(), words() & words() & words()))
        state["allowed"] = torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32)
    return state


def _run_logits(s):
    x = s["logits"]
    if own:
        from weight_streaming_expert_gb300 import adjust_logits
        return adjust_logits(x, history=s["history"], spans=s["spans"], repetition=s["repetition"],
                             presence=s["presence"], frequency=s["frequency"], bias_ids=s["bias_ids"],
                             bias_values=s["bias_values"], bias_starts=s["bias_starts"], allowed=s["allowed"])
    c, vocab = s["case"], x.shape[1]
    begin, answer, end = s["spans"].long()[:, :, None].unbind(1)
    at = begin + torch.arange(c["history"] + c["rows"], device=DEV)[None, :]
    token = s["history"].long()[at.clamp_max(s["history"].shape[0] - 1)]
    seen = torch.zeros_like(x).scatter_add_(1, token, (at < end).float()) > 0
    count = torch.zeros_like(x).scatter_add_(1, token, ((at < end) & (at >= answer)).float())
    rep = s["repetition"][:, None]
    x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
    x = x - s["frequency"][:, None] * count - s["presence"][:, None] * (count > 0)
    if s["bias_ids"] is not None:
        # of a row's entries for the same token the last one holds
        n = s["bias_ids"].shape[0]
        row = torch.searchsorted(s["bias_starts"].long(), torch.arange(n, device=DEV), right=True) - 1
        last = torch.full((x.numel(),), -1, dtype=torch.long, device=DEV)
        last = last.scatter_reduce_(0, row * vocab + s["bias_ids"].long(), torch.arange(n, device=DEV), "amax").view_as(x)
        x = x + torch.where(last >= 0, s["bias_values"][last.clamp_min(0)], torch.zeros_like(x))
    if s["allowed"] is not None:
        bit = torch.arange(vocab, device=DEV)
        x = torch.where((s["allowed"][:, bit // 32] >> (bit % 32).int()) & 1 != 0, x, -math.inf)
    return x


def _exact_logits(s):
    out = []
    for i, (begin, answer, end) in enumerate(s["spans"].tolist()):
        x = s["logits"][i].double()
        rep, presence, frequency = (float(s[n][i]) for n in ("repetition", "presence", "frequency"))
        prompt_and_answer = torch.unique(s["history"][begin:end].long())
        y = x[prompt_and_answer]
        x[prompt_and_answer] = torch.where(y > 0, y / rep, y * rep)
        made, times = torch.unique(s["history"][answer:end].long(), return_counts=True)
        x[made] -= presence + frequency * times.double()
        if s["bias_ids"] is not None:
            a, b = s["bias_starts"][i:i + 2].tolist()
            biases = dict(zip(s["bias_ids"][a:b].tolist(), s["bias_values"][a:b].tolist()))
            if biases:
                x[torch.tensor(list(biases), device=DEV)] += torch.tensor(list(biases.values()), dtype=torch.float64, device=DEV)
        if s["allowed"] is not None:
            bits = (s["allowed"][i].long()[:, None] >> torch.arange(32, device=DEV)) & 1
            x[bits.flatten()[:x.shape[0]] == 0] = -math.inf
        out.append(x)
    return torch.stack(out)


def exact(case, seed):
    return {"kv8": _exact_kv8, "attn": _exact_attn, "logits": _exact_logits}[case["op"]](prepare(case, seed))
