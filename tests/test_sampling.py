"""Sampling from logits (include/sampling.h).

Two references, neither of which shares the kernel's method (a full sort here):
`plain` follows the definition in whole numbers, with torch's fp32 exp, and has
to agree token by token; `exact` works with real numbers in 64 bits and says
for each row whether its outcome hangs on less than 2e-6 of the weights' sum
(every weight is off by at most (|z| + 2) 2^-23 for |z| up to 26, and as much
decides a border): rows that do not have to agree with it too."""
import math

import pytest
import torch

DEV = "cuda:0"
ONE = 1 << 38


def plain(x, u, t, k, p, least):
    """Token and probability of one row, x fp32 on the GPU."""
    x = torch.where(x.isnan(), torch.full_like(x, -math.inf), x)
    best, order = x.sort(descending=True, stable=True)
    if best[0] == -math.inf:
        return -1, 0.0
    if not t > 0:
        return int(order[0]), 1.0
    top = best[0]
    e = ((best - top) / torch.tensor(t, dtype=torch.float32, device=x.device)).exp()
    w = (torch.where(best == top, torch.ones_like(e), e) * ONE).long()
    w[(best == -math.inf) | e.isnan() & (best < top)] = 0  # infinitely far below, at any temperature
    n = len(w)
    if k > 0:
        w[k:] = 0
    if p < 1:
        before = w.cumsum(0) - w
        limit = float(torch.tensor(p, dtype=torch.float32)) * float(int(w.sum()))
        drop = before.double() >= limit
        drop[0] = False
        w[drop] = 0
    w[w.double() < min(float(torch.tensor(least, dtype=torch.float32)), 1.0) * ONE] = 0
    by_id = torch.zeros_like(w).scatter_(0, order, w)
    total = int(w.sum())
    wanted = min(int(float(u) * float(total)), total - 1)
    token = int((by_id.cumsum(0) <= wanted).sum())
    return token, int(by_id[token]) / total


def exact(x, u, t, k, p, least):
    """The same in real numbers; None where it hangs on too little."""
    close = 2e-6
    x = x.double().cpu()
    order = sorted(range(len(x)), key=lambda i: (-float(x[i]), i))
    z = x[order]
    w = torch.exp((z - z[0]) / t)
    if k > 0:
        order, w = order[:k], w[:k]
    if p < 1:
        cum = w.cumsum(0) / w.sum()
        n = int((cum < p).sum()) + 1
        if (cum - p).abs().min() < close:
            return None
        order, w = order[:n], w[:n]
    if least > 0:
        if (w / least - 1).abs().min() < 50 * close:
            return None
        order = [i for i, a in zip(order, w) if a >= least]
        w = w[w >= least]
    back = sorted(range(len(order)), key=lambda i: order[i])
    cum = w[back].cumsum(0) / w.sum()
    if len(back) > 1 and (cum[:-1] - u).abs().min() < close:
        return None
    at = min(int((cum <= u).sum()), len(back) - 1)
    return order[back[at]], float(w[back][at] / w.sum())


def logits(M, V, seed, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(M, V, generator=g) * spread + 6 * torch.rand(M, V, generator=g) ** 12).to(DEV)


def run(x, rows, u):
    from weight_streaming_expert_gb300 import sample
    col = lambda i, dt: torch.tensor([r[i] for r in rows], dtype=dt, device=DEV)
    tok, prob = sample(x, u.to(DEV), col(0, torch.float32), col(1, torch.int32), col(2, torch.float32),
                       col(3, torch.float32), return_probs=True)
    torch.cuda.synchronize()
    return tok.tolist(), prob.tolist()


SETTINGS = [(1.0, 0, 1.0, 0.0), (0.7, 50, 0.95, 0.02), (0.0, 0, 1.0, 0.0), (1.3, 0, 0.9, 0.0), (1.0, 1, 1.0, 0.0),
            (1.0, 0, 1.0, 0.1), (0.5, 7, 0.5, 0.0), (2.0, 1000, 0.999, 0.0), (1.0, 0, 0.0, 0.0), (1.0, 0, 1e-9, 0.0),
            (0.05, 3, 1.0, 0.0), (1.0, 10 ** 9, 1.0, 1.0), (30.0, 0, 0.3, 0.0)]


def check(x, rows, u, real=True):
    tok, prob = run(x, rows, u)
    decided = 0
    for i, (t, k, p, least) in enumerate(rows):
        want, want_p = plain(x[i], u[i], t, k, p, least)
        assert tok[i] == want, f"row {i} {rows[i]}: {tok[i]} instead of {want}"
        assert abs(prob[i] - want_p) <= 2.0 ** -23 * want_p
        if real and t > 0:
            r = exact(x[i], float(u[i]), t, k, p, least)
            if r is not None:
                decided += 1
                assert tok[i] == r[0] and abs(prob[i] - r[1]) <= 1e-5 * r[1]
    return decided


@pytest.mark.gpu
@pytest.mark.parametrize("V", [1, 2, 31, 32, 33, 100, 511, 512, 513, 1025, 4097, 8191])
def test_vocabularies(V):
    rows = [SETTINGS[i % len(SETTINGS)] for i in range(26)]
    u = torch.rand(26, generator=torch.Generator().manual_seed(V))
    decided = check(logits(26, V, V), rows, u)
    assert decided >= 16


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 6, 16, 64])
def test_model_vocabulary(M):
    rows = [SETTINGS[(i + M) % len(SETTINGS)] for i in range(M)]
    u = torch.rand(M, generator=torch.Generator().manual_seed(M))
    check(logits(M, 157184, M), rows, u, real=False)


@pytest.mark.gpu
def test_larger_vocabularies_and_many_rows():
    check(logits(2, 1_000_003, 1), SETTINGS[:2], torch.tensor([0.3, 0.8]), real=False)
    check(logits(1, 1 << 23, 4, spread=4.0), SETTINGS[3:4], torch.tensor([0.7]), real=False)
    rows = [SETTINGS[i % len(SETTINGS)] for i in range(700)]
    check(logits(700, 300, 2), rows, torch.rand(700, generator=torch.Generator().manual_seed(3)), real=False)


@pytest.mark.gpu
@pytest.mark.parametrize("V", [40960, 40961, 655360, 655361])
def test_where_a_slice_leaves_shared_memory(V):
    check(logits(len(SETTINGS), V, V), SETTINGS, torch.rand(len(SETTINGS), generator=torch.Generator().manual_seed(V)),
          real=False)
    # rows enough for one CTA each
    rows = [SETTINGS[i % len(SETTINGS)] for i in range(160)]
    if V < 50000:
        check(logits(160, V, V + 1), rows, torch.rand(160, generator=torch.Generator().manual_seed(1)), real=False)


@pytest.mark.gpu
@pytest.mark.parametrize("V", [512, 513, 2048, 2049, 20000])
@pytest.mark.parametrize("tied", [False, True])
def test_lengths_of_what_stays(V, tied):
    """Cuts on both sides of the lengths at which the kernel goes on another way."""
    rows = [(1.0, k, p, 0.0) for k in (2, 63, 64, 65, 511, 512, 513, 1024, 2047, 2048, 2049) for p in (1.0, 0.9, 0.2)]
    rows += [(t, 0, p, 0.0) for t in (0.5, 1.0, 4.0) for p in (0.1, 0.3, 0.5, 0.7, 0.99)]
    x = logits(len(rows), V, V)
    u = torch.rand(len(rows), generator=torch.Generator().manual_seed(V))
    check(x.round() if tied else x, rows, u, real=False)


@pytest.mark.gpu
def test_borders_of_the_uniform_number():
    x = torch.zeros(6, 1024, device=DEV)  # equal weights: token floor(u * 1024)
    u = torch.tensor([0.0, 1 / 1024, 0.5, 1 - 2.0 ** -24, 0.25 - 2.0 ** -26, 1.0])
    tok, prob = run(x, [(1.0, 0, 1.0, 0.0)] * 6, u)
    assert tok == [0, 1, 512, 1023, 255, 1023] and prob == [1 / 1024] * 6


@pytest.mark.gpu
@pytest.mark.parametrize("V", [64, 1000, 157184])
def test_ties_go_to_the_lower_id(V):
    g = torch.Generator().manual_seed(V)
    x = torch.randint(0, 4, (12, V), generator=g).float().to(DEV)
    x[3] = 0
    x[4, ::2], x[4, 1::2] = -0.0, 0.0
    rows = [(1.0, k, p, 0.0) for k in (1, 5, V // 3, V - 1) for p in (1.0, 0.6, 0.05)]
    check(x, rows, torch.rand(12, generator=g), real=False)


@pytest.mark.gpu
def test_infinities_nan_and_empty_rows():
    V = 700
    x = logits(9, V, 4)
    x[0] = -math.inf
    x[1] = math.nan
    x[2, 1:] = -math.inf
    x[3, ::2] = -math.inf
    x[4, [5, 600]] = math.inf
    x[5, 100:] = math.nan
    x[6] = -math.inf
    x[6, 699] = -3e38
    x[7] = 3e38
    x[7, 0] = -3e38
    x[8, 1::3] = math.inf
    x[8, ::3] = math.nan
    for row in SETTINGS:
        for u in (0.0, 0.37, 0.9999):
            check(x, [row] * 9, torch.full((9,), u), real=False)
    tok, prob = run(x[:2], [(1.0, 0, 1.0, 0.0), (0.0, 5, 0.5, 0.1)], torch.zeros(2))
    assert tok == [-1, -1] and prob == [0.0, 0.0]
    check(x, [(math.inf, 0, 1.0, 0.0)] * 9, torch.full((9,), 0.4), real=False)
    check(x, [(1e-30, 0, 0.9, 0.0)] * 9, torch.full((9,), 0.4), real=False)


@pytest.mark.gpu
def test_narrow_and_wide_logits():
    """Rows whose largest logits share their leading bits, or span all octaves."""
    g = torch.Generator().manual_seed(5)
    V = 5000
    x = torch.stack([100 + 1e-4 * torch.randn(V, generator=g), 1e-30 * torch.randn(V, generator=g),
                     torch.exp(40 * torch.randn(V, generator=g)).clamp(max=3e38), -1000 - torch.rand(V, generator=g),
                     torch.arange(V).float(), torch.full((V,), -0.0)]).to(DEV)
    for row in SETTINGS:
        check(x, [row] * 6, torch.rand(6, generator=g), real=False)


@pytest.mark.gpu
def test_frequencies_follow_the_probabilities():
    """20,000 draws of one row: chi-square over its 8 tokens (7 degrees of
    freedom: 40 is passed once in 10^6)."""
    p = torch.tensor([0.3, 0.05, 0.2, 0.1, 0.15, 0.08, 0.07, 0.05])
    x = p.log().to(DEV).expand(20000, 8)
    u = torch.rand(20000, generator=torch.Generator().manual_seed(6))
    tok, _ = run(x.contiguous(), [(1.0, 0, 1.0, 0.0)] * 20000, u)
    n = torch.bincount(torch.tensor(tok), minlength=8)
    assert float(((n - 20000 * p) ** 2 / (20000 * p)).sum()) < 40


@pytest.mark.gpu
def test_defaults_strides_and_given_tokens():
    from weight_streaming_expert_gb300 import sample
    x = logits(5, 1000, 7)
    u = torch.rand(5, generator=torch.Generator().manual_seed(8)).to(DEV)
    want = [plain(x[i], u[i], 1.0, 0, 1.0, 0.0)[0] for i in range(5)]
    assert sample(x, u).tolist() == want
    wide = torch.full((5, 1501), math.inf, device=DEV)
    wide[:, 300:1300] = x
    tokens = torch.zeros(5, dtype=torch.int32, device=DEV)
    assert sample(wide[:, 300:1300], u, tokens=tokens) is tokens and tokens.tolist() == want
    assert sample(x[:0], u[:0]).shape == (0,)


@pytest.mark.gpu
def test_graph_and_other_stream():
    from weight_streaming_expert_gb300 import sample
    x, u = logits(6, 20000, 9), torch.rand(6, generator=torch.Generator().manual_seed(10)).to(DEV)
    t = torch.full((6,), 0.8, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    sample(x, u, t, stream=s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        tok = sample(x, u, t, stream=s)
    for seed in (11, 12):
        x.copy_(logits(6, 20000, seed))
        g.replay()
        torch.cuda.synchronize()
        assert tok.tolist() == [plain(x[i], u[i], 0.8, 0, 1.0, 0.0)[0] for i in range(6)]


def test_refusals():
    import ctypes

    from weight_streaming_expert_gb300 import native as N
    L = N.lib()

    def call(logits=16, stride=100, rows=2, vocab=100, u=16, t=None, k=None, p=None, m=None, tokens=16, probs=None):
        v = lambda x: None if x is None else ctypes.c_void_p(x)
        return L.moe_sample(v(logits), stride, rows, vocab, v(u), v(t), v(k), v(p), v(m), v(tokens), v(probs), None)

    for bad in (dict(rows=-1), dict(rows=65536), dict(vocab=0), dict(vocab=(1 << 23) + 1), dict(logits=None),
                dict(u=None), dict(tokens=None), dict(logits=2), dict(t=1), dict(k=2), dict(p=3), dict(m=6),
                dict(probs=2), dict(stride=99)):
        assert call(**bad) == N.MOE_ERR_INVALID_ARG, bad
        assert N.last_error()
    assert call(rows=0, logits=None) == N.MOE_OK


@pytest.mark.gpu
def test_python_refusals():
    from weight_streaming_expert_gb300 import sample
    x, u = torch.zeros(2, 50, device=DEV), torch.zeros(2, device=DEV)
    for bad in (lambda: sample(x.half(), u), lambda: sample(x.cpu(), u), lambda: sample(x[0], u),
                lambda: sample(x, u[:1]), lambda: sample(x, u.double()), lambda: sample(x.T, u),
                lambda: sample(x, u, top_k=u), lambda: sample(x, u, temperature=torch.zeros(3, device=DEV)),
                lambda: sample(x, u, tokens=u)):
        with pytest.raises(ValueError):
            bad()
