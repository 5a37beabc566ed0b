"""Norms and rotation of queries and keys into the paged cache
(include/attention.h) against the formula in 64 bits.

Tolerance (h: half a step of the element type): one rounding of the result, h
|y|; before it fp32 arithmetic whose errors are relative to the pair: the sum
of D squares and its root (D/2 + 4) 2^-24, the products and the turn's sine and
cosine 16 * 2^-24 together, an angle off by 2^-25 half turns 2^-23: with D up to
256 less than 2^-16 of the pair's length.  fp16 results below its normal range
have a fixed half step of 2^-25."""
import math
from fractions import Fraction

import pytest
import torch

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


def turned(x, w, positions, rot, interleaved, eps, inv_freq):
    """x [T, H, D] in float64, and the length of each value's pair."""
    x = x.double()
    D = x.shape[2]
    if w is not None:
        x = x / torch.sqrt((x * x).mean(2, keepdim=True) + eps) * w.double()
    # the angle modulo a turn, from whole fractions
    angle = torch.tensor([[float(2 * PI * (Fraction(f) * p / (2 * PI) % 1)) for f in inv_freq] for p in positions],
                         dtype=torch.float64).view(len(positions), 1, -1)
    y, size = x.clone(), x.abs()
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        c, s = angle[..., i].cos(), angle[..., i].sin()
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., a] * s + x[..., b] * c
        size[..., a] = size[..., b] = torch.hypot(x[..., a], x[..., b])
    return y, size


def close(got, want, dtype):
    y, size = want
    h = torch.finfo(dtype).eps / 2
    tol = h * y.abs() + 2.0 ** -16 * size + (2.0 ** -25 if dtype == torch.float16 else 0)
    off = (got.cpu().double() - y).abs() - tol
    assert (off <= 0).all(), f"{off.max().item():.3g} past the bound"


def case(T, Hq, Hk, D, dtype, rot, interleaved, norm, page=16, far=100, seed=0, theta=10000.0, inv_freq=None):
    from weight_streaming_expert_gb300 import QKNormRope
    g = torch.Generator().manual_seed(seed)
    dt = TYPES[dtype]
    qkv = (torch.randn(T, Hq + 2 * Hk, D, generator=g) * 2).to(dt)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    qw = (1 + 0.3 * torch.randn(D, generator=g)).to(dt) if norm else None
    kw = (1 + 0.3 * torch.randn(D, generator=g)).to(dt) if norm else None
    positions = torch.randint(0, far + 1, (T,), generator=g).to(torch.int32)
    pages = T // page + 3
    slots = torch.randperm(pages * page, generator=g)[:T]
    slots[T // 2::5] = -1  # not kept
    kc = torch.randn(pages, page, Hk, D, generator=g).to(dt)
    vc = torch.randn(pages, page, Hk, D, generator=g).to(dt)
    op = QKNormRope(D, rotary_dim=rot, theta=theta, inv_freq=inv_freq, interleaved=interleaved, eps=1e-5, device=DEV)
    on = lambda t: None if t is None else t.to(DEV)
    x = on(qkv)
    kd, vd = on(kc), on(vc)
    out = op(x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:], on(qw), on(kw), on(positions), on(slots), kd, vd)
    freq = inv_freq or [theta ** (-2.0 * i / rot) for i in range(rot // 2)]
    pos = positions.tolist()
    close(out, turned(q, qw, pos, rot, interleaved, 1e-5, freq), dt)
    keep = slots >= 0
    y, size = turned(k, kw, pos, rot, interleaved, 1e-5, freq)
    rows = slots[keep]
    close(kd.flatten(0, 1)[rows.to(DEV)], (y[keep], size[keep]), dt)
    want_v = vc.clone()
    want_v.view(-1, Hk, D)[rows] = v[keep]
    assert torch.equal(vd.cpu(), want_v)
    others = torch.ones(pages * page, dtype=torch.bool)
    others[rows] = False
    assert torch.equal(kd.cpu().flatten(0, 1)[others], kc.flatten(0, 1)[others])


@pytest.mark.gpu
@pytest.mark.parametrize("D,rot", [(64, 64), (64, 32), (64, 16), (128, 128), (128, 64), (128, 112), (256, 256),
                                   (256, 48), (128, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_dims_and_pairings(D, rot, interleaved, dtype):
    case(5, 6, 2, D, dtype, rot, interleaved, norm=True, seed=D + rot)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (20, 4), (7, 1), (64, 8), (40, 40), (3, 3), (128, 2)])
@pytest.mark.parametrize("norm", [False, True])
def test_head_counts(Hq, Hk, norm):
    case(3, Hq, Hk, 128, "bf16", 128, False, norm, seed=Hq)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 2, 7, 64, 1000])
def test_token_counts(T):
    case(T, 4, 2, 64, "fp16", 64, False, True, seed=T)


@pytest.mark.gpu
@pytest.mark.parametrize("far", [1, 131072, 2 ** 31 - 1])
def test_far_positions(far):
    case(24, 4, 1, 128, "fp16", 128, True, True, far=far, seed=3, theta=1e6)
    case(24, 4, 1, 64, "bf16", 64, False, True, far=far, seed=4)


@pytest.mark.gpu
def test_given_frequencies():
    freq = [0.9 ** i * (3.0 if i % 3 else 0.01) for i in range(32)]
    case(9, 4, 2, 64, "bf16", 64, False, True, far=5000, inv_freq=freq)


@pytest.mark.gpu
def test_zero_row_and_in_place():
    from weight_streaming_expert_gb300 import QKNormRope
    op = QKNormRope(128, device=DEV)
    w = torch.ones(128, dtype=torch.bfloat16, device=DEV)
    q = torch.randn(4, 6, 128, device=DEV).bfloat16()
    q[2] = 0
    k = torch.zeros(4, 1, 128, dtype=torch.bfloat16, device=DEV)
    cache = [torch.full((2, 16, 1, 128), 3.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    pos = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device=DEV)
    slots = torch.tensor([0, 1, 2, 31], dtype=torch.int64, device=DEV)
    want = op(q, k, k, w, w, pos, slots, *cache)
    assert (want[2] == 0).all() and (cache[0].flatten(0, 1)[slots] == 0).all()
    got = op(q, k, k, w, w, pos, slots, *cache, q_out=q)
    assert got is q and torch.equal(q, want)


@pytest.mark.gpu
def test_slots_beyond_the_cache_write_nothing():
    from weight_streaming_expert_gb300 import QKNormRope
    op = QKNormRope(64, device=DEV)
    x = torch.randn(3, 2, 64, device=DEV).half()
    cache = [torch.full((4, 16, 2, 64), 3.0, dtype=torch.float16, device=DEV) for _ in range(2)]
    inner = [c[1:3] for c in cache]
    pos = torch.zeros(3, dtype=torch.int32, device=DEV)
    slots = torch.tensor([32, -1, 1 << 40], dtype=torch.int64, device=DEV)
    op(x, x, x, None, None, pos, slots, *inner)
    torch.cuda.synchronize()
    assert all((c == 3).all() for c in cache)


@pytest.mark.gpu
def test_graph_and_other_stream():
    from weight_streaming_expert_gb300 import QKNormRope
    op = QKNormRope(128, device=DEV)
    g0 = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(6, 24, 128, generator=g0, device=DEV).bfloat16()
    w = torch.ones(128, dtype=torch.bfloat16, device=DEV)
    pos = torch.arange(6, dtype=torch.int32, device=DEV)
    slots = torch.arange(6, device=DEV)
    cache = [torch.zeros(1, 16, 2, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    a = (x[:, :20], x[:, 20:22], x[:, 22:], w, w, pos, slots, *cache)
    want = op(*a).clone()
    kept = [c.clone() for c in cache]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = op(*a, stream=s)
    for c in cache:
        c.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and all(torch.equal(c, k) for c, k in zip(cache, kept))


def test_refusals():
    import ctypes

    from weight_streaming_expert_gb300 import native as N
    L = N.lib()
    base = dict(dtype=0, n_tokens=2, n_heads=4, n_kv_heads=2, head_dim=64, rotary_dim=64, interleaved=0, eps=1e-6,
                q=16, k=16, v=16, q_token_stride=256, q_head_stride=64, k_token_stride=128, k_head_stride=64,
                v_token_stride=128, v_head_stride=64, turns=16, positions=16, slots=16, q_out=16,
                q_out_token_stride=256, q_out_head_stride=64, k_cache=16, v_cache=16, k_page_stride=2048,
                k_row_stride=128, v_page_stride=2048, v_row_stride=128, n_pages=4, page_size=16)

    def call(**change):
        a = N.moe_qk_norm_rope_args_t()
        for k, v in {**base, **change}.items():
            setattr(a, k, v)
        return L.moe_qk_norm_rope(ctypes.byref(a), None)

    for bad in (dict(dtype=7), dict(n_tokens=-1), dict(rotary_dim=24), dict(rotary_dim=80), dict(rotary_dim=-16),
                dict(eps=-1.0), dict(eps=math.nan), dict(q=None), dict(q=8), dict(q_out=None), dict(k=None),
                dict(v_cache=4), dict(slots=None), dict(slots=4), dict(turns=None), dict(positions=2),
                dict(q_weight=8), dict(k_weight=2), dict(q_head_stride=60), dict(v_row_stride=4), dict(n_pages=0),
                dict(page_size=0)):
        assert call(**bad) == N.MOE_ERR_INVALID_ARG, bad
        assert N.last_error()
    assert call(head_dim=96) == N.MOE_ERR_UNSUPPORTED
    assert call(n_tokens=0, q=None) == N.MOE_OK
    assert L.moe_qk_norm_rope(None, None) == N.MOE_ERR_INVALID_ARG


def test_python_refusals():
    from weight_streaming_expert_gb300 import QKNormRope
    for bad in (dict(head_dim=80), dict(head_dim=64, rotary_dim=128), dict(head_dim=64, rotary_dim=8),
                dict(head_dim=64, inv_freq=[1.0]), dict(head_dim=64, rotary_dim=16, inv_freq=[math.inf] * 8)):
        with pytest.raises(ValueError):
            QKNormRope(**bad, device="cpu")


def test_turns_hold_the_angle_modulo_a_turn():
    from weight_streaming_expert_gb300 import QKNormRope
    op = QKNormRope(64, theta=10000.0, device="cpu")
    for i in (0, 1, 7, 31):
        for pos in (1, 12345, 2 ** 31 - 1):
            at = (int(op.turns[i]) * pos) % (1 << 64) / 2.0 ** 64
            want = float(Fraction(10000.0 ** (-2.0 * i / 64)) * pos / (2 * PI) % 1)
            off = abs(at - want)
            # the frequency's own rounding in 64 bits, over the position
            assert min(off, 1 - off) <= 2.0 ** -50 * pos * 10000.0 ** (-2.0 * i / 64) + 2.0 ** -30
