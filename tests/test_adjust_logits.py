"""Penalties, biases and masks on logits (include/sampling.h) against the
formula in 64 bits, token by token.

Tolerance (u = 2^-24): at most five fp32 operations in a row, each off by u of
its result.  With x0 the logit, r x0 or x0 / r after the first, and f c, p, b
the terms: every result along the way is at most S = max(|x0|, |x0| r, |x0| / r)
+ |f c| + |p| + |b|, the product f c one rounding more: 6 u S, and 1 % for what
the roundings do to one another."""
import math

import pytest
import torch

DEV = "cuda:0"
U = 2.0 ** -24


class Case:
    def __init__(self, M, V, spans=None, history=(), biases=None, mask=None, seed=0, penalties=(1.3, 0.4, 0.15)):
        g = torch.Generator().manual_seed(seed)
        self.logits = torch.randn(M, V, generator=g) * 3
        self.history, self.spans = torch.tensor(history, dtype=torch.int32), spans
        self.penalties = [None if p is None else p * (1 + 0.5 * torch.rand(M, generator=g)) for p in penalties]
        self.biases, self.mask = biases, mask  # lists of (token, bias) per row; rows of allowed tokens, None: all

    def inputs(self):
        on = lambda t: None if t is None else t.to(DEV)
        M, V = self.logits.shape
        x = dict(logits=on(self.logits), repetition=on(self.penalties[0]), presence=on(self.penalties[1]),
                 frequency=on(self.penalties[2]))
        if self.spans is not None:
            x.update(history=on(self.history), spans=torch.tensor(self.spans, dtype=torch.int32, device=DEV))
        if self.biases is not None:
            flat = [e for row in self.biases for e in row]
            starts = [0]
            for row in self.biases:
                starts.append(starts[-1] + len(row))
            x.update(bias_ids=torch.tensor([t for t, _ in flat], dtype=torch.int32, device=DEV),
                     bias_values=torch.tensor([b for _, b in flat], dtype=torch.float32, device=DEV),
                     bias_starts=torch.tensor(starts, dtype=torch.int32, device=DEV))
        if self.mask is not None:
            x["allowed"] = words_of(self.mask, V).to(DEV)
        return x

    def check(self, got):
        M, V = self.logits.shape
        got = got.cpu()
        for m in range(M):
            x = self.logits[m].double().clone()
            size = x.abs()
            rep, presence, frequency = (None if p is None else float(p[m]) for p in self.penalties)
            if self.spans is not None:
                n = len(self.history)
                begin, answer, end = self.spans[m]
                begin, end = max(begin, 0), min(end, n)
                inside = [int(t) for t in self.history[begin:end] if 0 <= t < V] if end > begin else []
                made = [int(t) for t in self.history[max(answer, begin):end] if 0 <= t < V] if end > max(answer, begin) else []
                if rep is not None:
                    for t in set(inside):
                        x[t] = x[t] / rep if x[t] > 0 else x[t] * rep
                        size[t] = size[t] * max(rep, 1 / rep, 1)
                for t in set(made):
                    for d in ((frequency or 0) * made.count(t), presence or 0):
                        x[t] -= d
                        size[t] += abs(d)
            if self.biases is not None:
                for t, b in dict(self.biases[m]).items():
                    if 0 <= t < V:
                        x[t] += float(torch.tensor(b, dtype=torch.float32))
                        size[t] += abs(b)
            if self.mask is not None and self.mask[m] is not None:
                hidden = torch.ones(V, dtype=torch.bool)
                hidden[list(self.mask[m])] = False
                x[hidden] = -math.inf
            fine = x > -math.inf
            assert torch.equal(got[m] == -math.inf, ~fine)
            assert ((got[m].double() - x).abs()[fine] <= 6.06 * U * size[fine]).all(), f"row {m}"


def words_of(mask, V):
    words = torch.zeros(len(mask), -(-V // 32), dtype=torch.int64)
    for m, row in enumerate(mask):
        if row is None:
            words[m] = 0xffffffff
        else:
            for t in row:
                words[m, t // 32] |= 1 << (t % 32)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)


def run(case, **more):
    from weight_streaming_expert_gb300 import adjust_logits
    x = case.inputs()
    x.update(more)
    before = x["logits"].clone()
    got = adjust_logits(**x)
    case.check(got)
    assert torch.equal(before, x["logits"])
    again = x["logits"].clone()
    assert adjust_logits(**{**x, "logits": again, "out": again}) is again
    assert torch.equal(again, got)  # in place: the same bits
    return got


def mixed(M, V, seed, length=50):
    g = torch.Generator().manual_seed(seed)
    r = lambda n: [int(t) for t in torch.randint(0, V, (n,), generator=g)]
    history = [t % max(1, V // 3) for t in r(M * length)]
    spans = [(m * length, m * length + length // 3, (m + 1) * length) for m in range(M)]
    biases = [[(t, 0.5 * i - 3) for i, t in enumerate(r(m % 7))] for m in range(M)]
    mask = [None if m % 3 == 0 else sorted(set(r(max(1, V // 2)))) for m in range(M)]
    return Case(M, V, spans, history, biases, mask, seed)


@pytest.mark.gpu
@pytest.mark.parametrize("V", [1, 2, 3, 4, 5, 31, 32, 33, 63, 100, 4093, 4096, 4097, 8190, 12345])
def test_vocabularies(V):
    run(mixed(5, V, seed=V))


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 2, 64, 300])
def test_rows(M):
    run(mixed(M, 777, seed=M, length=20))


@pytest.mark.gpu
def test_each_part_alone_and_nothing():
    c = mixed(4, 5000, seed=1)
    for part in ("rep", "presence", "frequency", "bias", "mask", "none", "counts without penalties"):
        d = mixed(4, 5000, seed=1)
        d.penalties = [p if part == n else None for p, n in zip(c.penalties, ("rep", "presence", "frequency"))]
        if part not in ("rep", "presence", "frequency", "counts without penalties"):
            d.spans = None
        d.biases = c.biases if part == "bias" else None
        d.mask = c.mask if part == "mask" else None
        got = run(d)
        if part in ("none", "counts without penalties"):
            assert torch.equal(got.cpu(), c.logits)


@pytest.mark.gpu
def test_repeats_shared_spans_and_strangers():
    # rows of one chain; the same token many times; tokens outside the vocabulary; spans past the history
    history = [7] * 1000 + [8, 7, 99, 98] + [-1, 1 << 30, 100, -(1 << 31)] + [3]
    n = len(history)
    spans = [(0, 1000, n - 1), (0, 1000, n), (0, 0, n), (-5, -3, n + 100), (n, n, n), (5, 2, 3), (0, n + 7, n)]
    run(Case(7, 100, spans, history, seed=2))


@pytest.mark.gpu
def test_of_several_biases_the_last_holds():
    rows = [[(5, 1.0), (5, 2.0), (5, -7.0)], [], [(i % 10, float(i)) for i in range(1000)], [(-1, 9.0), (300, 9.0)]]
    got = run(Case(4, 300, biases=rows, seed=3))
    case = Case(4, 300, biases=rows, seed=3)
    assert got[0, 5].item() == pytest.approx(case.logits[0, 5].item() - 7.0, rel=1e-6)


@pytest.mark.gpu
def test_bias_starts_are_cut_to_the_list():
    from weight_streaming_expert_gb300 import adjust_logits
    x = torch.zeros(3, 40, device=DEV)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)
    got = adjust_logits(x, bias_ids=i32(1, 2, 3), bias_values=torch.tensor([1.0, 2.0, 3.0], device=DEV),
                        bias_starts=i32(-9, 2, 100, 1)).cpu()
    want = torch.zeros(3, 40)
    want[0, 1], want[0, 2], want[1, 3] = 1.0, 2.0, 3.0
    assert torch.equal(got, want)


@pytest.mark.gpu
def test_masks_that_leave_nothing_or_one_token():
    from weight_streaming_expert_gb300 import sample
    c = Case(3, 1000, mask=[[], [999], [0]], seed=4)
    got = run(c)
    assert sample(got, torch.full((3,), 0.5, device=DEV)).tolist() == [-1, 999, 0]
    shared = c.inputs()["allowed"][1:2].expand(3, -1)
    c.mask = [[999]] * 3
    run(c, allowed=shared)


@pytest.mark.gpu
def test_infinities_and_nan():
    from weight_streaming_expert_gb300 import adjust_logits
    nan, inf = math.nan, math.inf
    x = torch.tensor([[nan, inf, -inf, nan, inf, -inf, 0.0, -0.0]], device=DEV)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)
    got = adjust_logits(x, history=i32(0, 1, 2, 6, 7), spans=i32(0, 0, 5).view(1, 3), repetition=torch.tensor([2.0], device=DEV),
                        presence=torch.tensor([0.5], device=DEV), allowed=i32(0b11100111).view(1, 1)).tolist()[0]
    assert math.isnan(got[0]) and got[1:] == [inf, -inf, -inf, -inf, -inf, -0.5, -0.5]


@pytest.mark.gpu
@pytest.mark.parametrize("offset,wide", [(0, 5003), (1, 5004), (2, 5001), (3, 6000)])
def test_strided_and_misaligned_rows(offset, wide):
    c = mixed(4, 5000, seed=5)
    buf = torch.zeros(4, wide + 4, device=DEV)
    x = c.inputs()
    view = buf[:, offset:offset + 5000]
    view.copy_(x["logits"])
    whole = torch.full((4, 5010), 42.0, device=DEV)
    from weight_streaming_expert_gb300 import adjust_logits
    for out in (None, whole[:, 3:5003], whole[:, offset:offset + 5000]):
        whole.fill_(42.0)
        got = adjust_logits(**{**x, "logits": view, "out": out})
        c.check(got)
        if out is not None:
            first = out.storage_offset()
            assert (whole[:, :first] == 42).all() and (whole[:, first + 5000:] == 42).all()
    adjust_logits(**{**x, "logits": view, "out": view})
    c.check(view)
    assert (buf[:, :offset] == 0).all() and (buf[:, offset + 5000:] == 0).all()


@pytest.mark.gpu
def test_expanded_logits():
    from weight_streaming_expert_gb300 import adjust_logits
    c = mixed(3, 900, seed=6)
    one = c.logits[:1].clone()
    c.logits = one.expand(3, -1)
    x = c.inputs()
    c.check(adjust_logits(**{**x, "logits": one.to(DEV).expand(3, -1)}))


@pytest.mark.gpu
def test_long_histories_and_large_vocabularies():
    run(mixed(3, 157184, seed=7, length=3000))


@pytest.mark.gpu
def test_rows_beyond_32_bit_offsets():
    from weight_streaming_expert_gb300 import adjust_logits
    c = mixed(3, 700, seed=10)
    x = c.inputs()
    far = torch.empty(2 * ((1 << 30) + 700) + 700, device=DEV)  # rows 2^32 bytes apart and more
    view = far.as_strided((3, 700), ((1 << 30) + 700, 1))
    view.copy_(x["logits"])
    c.check(adjust_logits(**{**x, "logits": view}))
    adjust_logits(**{**x, "logits": view, "out": view})
    c.check(view)


@pytest.mark.gpu
def test_captured_and_on_another_stream():
    from weight_streaming_expert_gb300 import adjust_logits
    c = mixed(6, 3001, seed=8)
    x = c.inputs()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = adjust_logits(**x, stream=side)
    side.synchronize()
    c.check(got)
    out = torch.empty_like(got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        adjust_logits(**x, out=out)
    d = mixed(6, 3001, seed=9)
    for name, t in d.inputs().items():
        if name in ("logits", "history", "spans", "repetition", "presence", "frequency", "allowed"):
            x[name].copy_(t)
    d.biases = c.biases
    graph.replay()
    torch.cuda.synchronize()
    d.check(out)


@pytest.mark.gpu
def test_no_rows_and_empty_lists():
    from weight_streaming_expert_gb300 import adjust_logits
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=DEV)
    assert adjust_logits(torch.zeros(0, 10, device=DEV)).shape == (0, 10)
    x = torch.randn(2, 10, device=DEV)
    got = adjust_logits(x, history=i32(0), spans=i32(2, 3), repetition=torch.full((2,), 2.0, device=DEV), bias_ids=i32(0),
                        bias_values=torch.zeros(0, device=DEV), bias_starts=i32(3))
    assert torch.equal(got, x)


def good_call(dev):
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=dev)
    f = lambda *s: torch.zeros(*s, device=dev)
    return dict(logits=f(2, 40), history=i32(5), spans=i32(2, 3), repetition=f(2), presence=f(2), frequency=f(2),
                bias_ids=i32(4), bias_values=f(4), bias_starts=i32(3), allowed=i32(2, 2), out=f(2, 40))


@pytest.mark.gpu
def test_refusals():
    from weight_streaming_expert_gb300 import adjust_logits
    good = good_call(DEV)
    adjust_logits(**good)
    for name, t in good.items():
        bads = [[1.0], 3, t.double(), t.cpu(), t[..., None], t[..., :-1] if name not in ("history",) else t[::2]]
        if name not in ("repetition", "presence", "frequency", "allowed", "out"):
            bads.append(None)
        for bad in bads:
            if name == "logits" and isinstance(bad, torch.Tensor) and bad.dtype == torch.float32 and bad.is_cuda and bad.dim() == 2:
                continue  # a narrower vocabulary: the others do not fit it then
            if name in ("bias_ids", "bias_values") and isinstance(bad, torch.Tensor) and bad.dim() == 1 and bad.is_cuda and bad.dtype == t.dtype:
                with pytest.raises(ValueError, match="bias_values"):
                    adjust_logits(**{**good, name: bad})
                continue
            with pytest.raises(ValueError, match="history|spans" if name in ("history", "spans") else
                               "bias_" if name.startswith("bias") else name):
                adjust_logits(**{**good, name: bad})


def test_refusals_on_the_cpu():
    from weight_streaming_expert_gb300 import adjust_logits
    with pytest.raises(ValueError, match="logits"):
        adjust_logits(**good_call("cpu"))
    for bad in (None, [1.0], torch.zeros(3)):
        with pytest.raises(ValueError, match="logits"):
            adjust_logits(bad)


def test_c_call_refuses_before_the_gpu():
    import ctypes

    from weight_streaming_expert_gb300 import native as N
    L = N.lib()

    def call(**k):
        a = N.moe_adjust_logits_args_t(logits=4096, row_stride=64, out=8192, out_stride=64, rows=2, vocab=64)
        for name, v in k.items():
            setattr(a, name, v)
        return L.moe_adjust_logits(ctypes.byref(a), None)

    assert L.moe_adjust_logits(None, None) == N.MOE_ERR_INVALID_ARG
    assert call(rows=0) == N.MOE_OK
    for bad, text in ((dict(rows=-1), "rows"), (dict(rows=65536), "rows"), (dict(vocab=0), "vocab"),
                      (dict(vocab=8388609), "vocab"), (dict(logits=None), "null"), (dict(out=8193), "aligned"),
                      (dict(history=4096), "spans"), (dict(bias_ids=4096), "bias_values"), (dict(allowed=2), "aligned"),
                      (dict(out_stride=63), "overlap"), (dict(row_stride=-1), "strides"), (dict(n_history=-1), "n_history"),
                      (dict(out=4096, out_stride=128), "in place"), (dict(allowed_stride=-1), "allowed_stride")):
        assert call(**bad) == N.MOE_ERR_INVALID_ARG, bad
        assert text in N.last_error(), (bad, N.last_error())
