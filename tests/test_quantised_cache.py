"""The quantised cache (include/attention.h): E4M3 codes with a power of two for
each row of a head, written by QKNormRope, read back by read_cache and moved by
PagedKVCache.

What is not computed on the way is compared bit by bit with the definition in
plain operations: values, and keys without norm and rotation.  Keys with them
are off before the codes by less than 2^-16 of their pair's length (the bound
that test_qk_norm_rope derives), so the exponent is that of a largest value
within 2^-16 of the true one, and a code within half a step (2^-4 of itself, or
2^-10) and that error of the true value."""
import math

import pytest
import torch

from tests.test_qk_norm_rope import TYPES, close, turned

DEV = "cuda:0"
E4M3 = torch.float8_e4m3fn


def exponent(largest):
    mantissa, e = torch.frexp(largest)
    e = torch.where(largest > 0, e - torch.where(mantissa <= 0.875, 9, 8), -40)  # the least of all for 0
    return e.clamp(-40, 40)


def quantised(x):
    """Codes (as bytes) and exponents of rows [..., D] of fp32 values."""
    size = torch.where(x.abs() < math.inf, x.abs(), torch.zeros_like(x))
    e = exponent(size.amax(-1))
    y = torch.ldexp(x.double(), -e[..., None]).clamp(-448, 448).float()
    y = torch.where(x.abs() == math.inf, torch.full_like(y, math.nan), y)
    return y.to(E4M3).view(torch.uint8), e


def same_codes(got, want):
    """Bit by bit, where any NaN is as good as another."""
    nan = lambda t: (t & 0x7f) == 0x7f
    return torch.equal(nan(got), nan(want)) and torch.equal(got[~nan(got)], want[~nan(want)])


def empty_cache(pages, page, Hk, D, fill=0x5a, scale=99):
    b = lambda *s, v: torch.full(s, v, dtype=torch.uint8, device=DEV)
    return dict(k_cache=b(pages, page, Hk, D, v=fill).view(E4M3), v_cache=b(pages, page, Hk, D, v=fill).view(E4M3),
                k_scale=b(pages, Hk, page, v=scale), v_scale=b(pages, Hk, page, v=scale))


def rows_of(cache, name):
    """Codes [slots, Hk, D] and scale bytes [slots, Hk]."""
    return (cache[name + "_cache"].view(torch.uint8).flatten(0, 1).cpu(),
            cache[name + "_scale"].transpose(1, 2).flatten(0, 1).cpu())


def write(x, Hq, Hk, D, cache, slots, positions=None, rot=0, qw=None, kw=None, **op):
    from weight_streaming_expert_gb300 import QKNormRope
    x = x.to(DEV)
    positions = torch.zeros(x.shape[0], dtype=torch.int32) if positions is None else positions
    on = lambda t: None if t is None else t.to(DEV)
    return QKNormRope(D, rotary_dim=rot, device=DEV, **op)(
        x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:], on(qw), on(kw), positions.to(DEV), slots.to(DEV), **cache)


def case(T, Hq, Hk, D, dtype, rot, interleaved, norm, page=16, seed=0):
    g = torch.Generator().manual_seed(seed)
    dt = TYPES[dtype]
    qkv = (torch.randn(T, Hq + 2 * Hk, D, generator=g) * 2).to(dt)
    qkv[:, Hq:] *= torch.exp2(torch.randint(-6, 7, (T, 2 * Hk, 1), generator=g).float()).to(dt)
    weight = lambda: (1 + 0.3 * torch.randn(D, generator=g)).to(dt) if norm else None
    qw, kw = weight(), weight()
    positions = torch.randint(0, 100000, (T,), generator=g).to(torch.int32)
    pages = T // page + 3
    slots = torch.randperm(pages * page, generator=g)[:T]
    slots[T // 2::5] = -1  # not kept
    cache = empty_cache(pages, page, Hk, D)
    op = dict(interleaved=interleaved, eps=1e-5, theta=1e5)
    q = write(qkv, Hq, Hk, D, cache, slots, positions, rot, qw, kw, **op)
    freq = [1e5 ** (-2.0 * i / rot) for i in range(rot // 2)]
    close(q, turned(qkv[:, :Hq], qw, positions.tolist(), rot, interleaved, 1e-5, freq), dt)
    keep = slots >= 0
    rows = slots[keep]
    codes, scale = rows_of(cache, "v")
    want, e = quantised(qkv[keep, Hq + Hk:].float())
    assert same_codes(codes[rows], want) and torch.equal(scale[rows].int() - 127, e)
    y, size = turned(qkv[:, Hq:Hq + Hk], kw, positions.tolist(), rot, interleaved, 1e-5, freq)
    y, size = y[keep], size[keep]
    codes, scale = rows_of(cache, "k")
    got_e = scale[rows].int() - 127
    largest = y.abs().amax(-1)
    slack = (size.amax(-1) * 2.0 ** -16)
    assert (got_e >= exponent((largest - slack).clamp_min(0))).all() and (got_e <= exponent(largest + slack)).all()
    got = codes[rows].view(E4M3).double()
    unit = torch.exp2(got_e.double())[..., None]
    x = y / unit
    off = (got - x).abs() - (x.abs() * 2.0 ** -4).clamp_min(2.0 ** -10) - 1.1 * 2.0 ** -16 * size / unit
    assert (off <= 0).all(), f"{off.max().item():.3g} past the bound"
    others = torch.ones(pages * page, dtype=torch.bool)
    others[rows] = False
    for name in "kv":
        codes, scale = rows_of(cache, name)
        assert (codes[others] == 0x5a).all() and (scale[others] == 99).all()


@pytest.mark.gpu
@pytest.mark.parametrize("D,rot", [(64, 64), (64, 32), (128, 128), (128, 48), (128, 0), (256, 256)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_written_rows(D, rot, interleaved, dtype):
    case(13, 6, 2, D, dtype, rot, interleaved, norm=True, seed=D + rot)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (20, 4), (7, 1), (64, 8), (3, 3), (0, 5), (128, 2)])
def test_head_counts(Hq, Hk):
    case(5, Hq, Hk, 128, "bf16", 128, False, norm=False, seed=Hq)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 2, 63, 700, 6000])
def test_token_counts(T):
    case(T, 4, 2, 64, "fp16", 64, False, True, page=32, seed=T)


def special_rows(dt, D):
    """Rows whose largest value stands at a border of the scales, rows of ties,
    nothing, infinities, NaN, and values beyond both ends."""
    g = torch.Generator().manual_seed(5)
    rows = [torch.zeros(D)]
    base = (torch.rand(D, generator=g) * 2 - 1)
    top = 2.0 ** 14 if dt == torch.float16 else 2.0 ** 60
    step = torch.finfo(dt).eps
    for largest in (448.0, 448.0 * (1 + step), 448 * (1 - step), 1.75, 1.75 * (1 + 2 * step), 224.0, 2.0 ** -14, top, 1.0):
        r = base * largest
        r[3] = -largest
        rows.append(r)
    ties = torch.arange(D).float() / 32 + 8  # every second one between two codes
    ties[0] = 448.0
    rows.append(ties)
    for bad in (math.nan, math.inf, -math.inf):
        r = base * 3
        r[1] = bad
        rows.append(r)
    rows.append(torch.full((D,), math.nan))
    rows.append(torch.full((D,), math.inf))
    if dt == torch.bfloat16:
        rows += [base * 2.0 ** -60, base * 2.0 ** -48, base * 1e-38, base * 3e38]
    return torch.stack(rows).to(dt)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_borders_infinities_and_nan(D, dtype):
    from weight_streaming_expert_gb300 import read_cache
    rows = special_rows(TYPES[dtype], D)
    T = rows.shape[0]
    x = torch.stack((rows, rows.flip(0)), 1)  # one key and one value head, no queries
    cache = empty_cache(4, 16, 1, D)
    slots = torch.arange(T)
    write(x, 0, 1, D, cache, slots)
    for name, y in (("k", x[:, :1]), ("v", x[:, 1:])):
        codes, scale = rows_of(cache, name)
        want, e = quantised(y.float())
        assert same_codes(codes[:T], want) and torch.equal(scale[:T].int() - 127, e)
    for got, y in zip(read_cache(**cache, slots=slots.to(DEV)), (x[:, :1], x[:, 1:])):
        codes, e = quantised(y.float())
        want = torch.ldexp(codes.view(E4M3).float(), e[..., None])
        assert torch.equal(got.cpu().isnan(), want.isnan())
        assert torch.equal(got.cpu().float().nan_to_num(7.0), want.nan_to_num(7.0))


@pytest.mark.gpu
@pytest.mark.parametrize("Hk,D,page", [(1, 64, 16), (4, 128, 64), (3, 256, 32), (8, 128, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_reading_back(Hk, D, page, dtype):
    """Every code under scales of every kind, unused ones among them."""
    from weight_streaming_expert_gb300 import read_cache
    g = torch.Generator().manual_seed(Hk)
    pages, dt = 300 // page + 2, TYPES[dtype]
    cache = empty_cache(pages, page, Hk, D)
    for name in "kv":
        cache[name + "_cache"].view(torch.uint8).copy_(torch.randint(0, 256, (pages, page, Hk, D), generator=g))
        cache[name + "_scale"].copy_(torch.randint(80, 175, (pages, Hk, page), generator=g))
    cache["k_scale"][0] = torch.tensor([0, 255, 87, 167] * (-(-Hk * page // 4)), dtype=torch.uint8)[:Hk * page].view(Hk, page)
    total = pages * page
    slots = torch.randint(-2, total + 2, (301,), generator=g)
    slots[:4] = torch.tensor([-1, total, 1 << 60, -(1 << 62)])
    got = read_cache(**cache, slots=slots.to(DEV), dtype=dt)
    for name, out in zip("kv", got):
        codes, scale = rows_of(cache, name)
        inside = (slots >= 0) & (slots < total)
        at = slots.clamp(0, total - 1)
        want = torch.ldexp(codes[at].view(E4M3).double(), (scale[at].int() - 127).clamp(-40, 40)[..., None])
        want = torch.where(inside[:, None, None], want, torch.zeros_like(want))
        if dtype == "fp16":
            want = want.clamp(-65504, 65504)
        want = want.float().to(dt)  # fp32 holds every one of them
        assert torch.equal(out.cpu().isnan(), want.isnan())
        assert torch.equal(out.cpu().nan_to_num(7.0), want.nan_to_num(7.0))


@pytest.mark.gpu
def test_reading_into_strided_outputs_and_of_nothing():
    from weight_streaming_expert_gb300 import read_cache
    cache = empty_cache(3, 16, 2, 64, fill=0x38, scale=128)  # ones times two
    slots = torch.arange(20, device=DEV)
    wide = torch.full((20, 5, 80), 9.0, device=DEV).bfloat16()
    k, v = read_cache(**cache, slots=slots, k_out=wide[:, 1:3, :64], v_out=wide[:, 3:5, 16:])
    assert k.data_ptr() == wide[:, 1:3].data_ptr() and (k == 2).all() and (v == 2).all()
    assert (wide[:, 0] == 9).all() and (wide[:, 1:3, 64:] == 9).all() and (wide[:, 3:, :16] == 9).all()
    assert read_cache(**cache, slots=slots[:0])[0].shape == (0, 2, 64)


@pytest.mark.gpu
def test_write_and_read_captured():
    from weight_streaming_expert_gb300 import QKNormRope, read_cache
    x = torch.randn(4, 6, 128, device=DEV).half()
    cache = empty_cache(2, 16, 2, 128)
    op, slots = QKNormRope(128, device=DEV), torch.arange(4, device=DEV)
    pos = torch.arange(4, device=DEV, dtype=torch.int32)
    step = lambda: (op(x[:, :2], x[:, 2:4], x[:, 4:], None, None, pos, slots, **cache),
                    *read_cache(**cache, slots=slots, dtype=torch.float16))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    x.copy_(torch.randn_like(x) * 3)
    pos += 1000
    slots += 9
    graph.replay()
    want = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, want))


@pytest.mark.gpu
@pytest.mark.parametrize("Hk,page", [(1, 16), (2, 32), (4, 64)])
def test_scales_move_with_their_rows(Hk, page):
    """Forks, copies on write, the accepted rows of trees and compaction: each
    sequence reads back what was written for it."""
    import random

    from weight_streaming_expert_gb300 import PagedKVCache, read_cache
    rng = random.Random(page)
    cache = PagedKVCache(2, 40, page, Hk, 64, 12 * page, dtype=E4M3, device=DEV)
    g = torch.Generator().manual_seed(1)
    model = {}  # sequence -> [n, layers, 2, Hk, D] in bf16, on powers of two and codes: exact

    def new_rows(n):
        codes = torch.randint(0, 0x7f, (n, 2, 2, Hk, 64), generator=g).to(torch.uint8).view(E4M3).float()
        codes[..., 0] = 448.0  # the scale is the exponent
        return torch.ldexp(codes, torch.randint(-20, 20, (n, 2, 2, Hk, 1), generator=g)).bfloat16()

    def extend(s, n):
        slots, rows = cache.extend(s, n), new_rows(n)
        for layer in range(2):
            write(torch.cat((rows[:, layer, 0], rows[:, layer, 1]), 1), 0, Hk, 64, cache.layer(layer), slots)
        model[s] = torch.cat((model[s], rows))

    for _ in range(3):
        s = cache.open()
        model[s] = new_rows(0)
        extend(s, rng.randint(1, 2 * page))
    for step in range(30):
        s = rng.choice(list(model))
        act = rng.choice(["extend", "fork", "keep", "keep", "compact", "free"])
        if act == "extend" and cache.length(s) < 9 * page and cache.table.free_pages > 6:
            extend(s, rng.randint(1, page))
        elif act == "fork" and len(model) < 6 and cache.table.free_pages > 6:
            model[cache.fork(s)] = model[s].clone()
        elif act == "keep" and cache.length(s) > 4 and cache.table.free_pages > 6:
            n = cache.length(s)
            start = rng.randint(max(0, n - 70), n - 2)
            accepted = sorted(rng.sample(range(n - start), rng.randint(1, n - start)))
            cache.keep(s, start, accepted)
            model[s] = torch.cat((model[s][:start], model[s][[start + i for i in accepted]]))
        elif act == "compact":
            cache.compact()
        elif act == "free" and len(model) > 2:
            cache.free(s)
            del model[s]
        for s, rows in model.items():
            slots = torch.tensor(cache.table.slots(s, range(cache.length(s))), dtype=torch.int64, device=DEV)
            for layer in range(2):
                k, v = read_cache(**cache.layer(layer), slots=slots)
                assert torch.equal(k.cpu(), rows[:, layer, 0]) and torch.equal(v.cpu(), rows[:, layer, 1])


@pytest.mark.gpu
def test_pages_whose_scales_do_not_fit_are_refused_before_any_moves():
    from weight_streaming_expert_gb300 import copy_pages
    pools = {n: torch.zeros(1, 4, 8, 1, 64, dtype=torch.uint8, device=DEV) for n in ("k_pool", "v_pool")}
    pools["k_pool"][:, 0] = 7
    scale = torch.zeros(1, 4, 1, 8, dtype=torch.uint8, device=DEV)
    i = torch.arange(2, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError, match="16 bytes"):
        copy_pages(**pools, src=i[:1], dst=i[1:], k_scale=scale, v_scale=scale.clone())
    assert (pools["k_pool"][:, 1] == 0).all()


@pytest.mark.gpu
def test_codes_beyond_32_bit_offsets():
    """Rows past 2^32 bytes of the pool, written, read back and attended to."""
    from weight_streaming_expert_gb300 import PagedAttention, read_cache
    page, Hk, D = 256, 8, 128
    pages = (1 << 32) // (page * Hk * D) + 9
    cache = {n + "_cache": torch.empty(pages, page, Hk, D, dtype=torch.uint8, device=DEV).view(E4M3) for n in "kv"}
    cache.update({n + "_scale": torch.empty(pages, Hk, page, dtype=torch.uint8, device=DEV) for n in "kv"})
    x = torch.randn(300, 3 * Hk, D, generator=torch.Generator().manual_seed(1)).bfloat16()
    table = torch.tensor([[pages - 1, pages - 3]], dtype=torch.int32)
    at = torch.arange(300)
    slots = table[0].long()[at // page] * page + at % page
    q = write(x, Hk, Hk, D, cache, slots)
    k, v = read_cache(**cache, slots=slots.to(DEV))
    for got, y in ((k, x[:, Hk:2 * Hk]), (v, x[:, 2 * Hk:])):
        codes, e = quantised(y.float())
        assert torch.equal(got.cpu().float(), torch.ldexp(codes.view(E4M3).float(), e[..., None]))
    attn = PagedAttention(Hk, Hk, D, device=DEV)
    i32 = lambda *t: torch.tensor(t, dtype=torch.int32, device=DEV)
    for m in (1, 90):  # over the codes, and through 16 bits
        out = attn(q[300 - m:], block_table=table.to(DEV), q_starts=i32(0, m), kv_lens=i32(300), max_q_len=m, **cache)
        s = torch.einsum("mhd,nhd->hmn", q[300 - m:].double(), k.double()) * D ** -0.5
        s.masked_fill_(torch.arange(300, device=DEV)[None, None] > (300 - m + torch.arange(m, device=DEV))[None, :, None], -math.inf)
        want = torch.einsum("hmn,nhd->mhd", s.softmax(-1), v.double())
        # two roundings to bf16, relative to values of at most the largest
        assert (out.double() - want).abs().max() <= 2.0 ** -7 * v.abs().max()
    assert attn.status() == 0
    attn.close()


@pytest.mark.gpu
def test_refusals():
    from weight_streaming_expert_gb300 import QKNormRope, copy_pages, copy_rows, read_cache
    cache = empty_cache(3, 16, 2, 64)
    x = torch.zeros(2, 2, 64, device=DEV).half()
    i = torch.arange(2, device=DEV)
    op = QKNormRope(64, device=DEV)
    good = dict(q=x, k=x, v=x, q_weight=None, k_weight=None, positions=i.int(), slots=i, **cache)
    op(**good)
    read = dict(**cache, slots=i, k_out=x, v_out=x.clone(), dtype=torch.float16)
    read_cache(**read)
    for call, kwargs in ((op, good), (read_cache, read)):
        for name in ("k_cache", "v_cache"):
            for bad in (cache[name].view(torch.uint8), cache[name].view(torch.uint8).half(),
                        cache[name].view(torch.uint8)[..., :32].view(E4M3), 3):
                with pytest.raises(ValueError, match="k_cache|v_cache"):
                    call(**{**kwargs, name: bad})
        for name in ("k_scale", "v_scale"):
            for bad in (cache[name].float(), cache[name][:, :1], cache[name].transpose(1, 2), cache[name].cpu(),
                        None, "x"):
                with pytest.raises(ValueError, match="k_scale|v_scale"):
                    call(**{**kwargs, name: bad})
    for name in ("k_out", "v_out"):
        for bad in (x[:1], x.float(), x[..., :32]):
            with pytest.raises(ValueError, match="k_out|v_out|outputs"):
                read_cache(**{**read, name: bad})
    with pytest.raises(ValueError, match="dtype"):
        read_cache(**{**read, "dtype": torch.float32})
    for bad in (i.int(), i[:, None], None):
        with pytest.raises(ValueError, match="slots"):
            read_cache(**{**read, "slots": bad})
    pools = dict(k_pool=cache["k_cache"][None], v_pool=cache["v_cache"][None], src=i[:1], dst=i[1:])
    for call in (copy_pages, copy_rows):
        pages = dict(pools, src=i[:1].int(), dst=i[1:].int()) if call is copy_pages else pools
        scales = dict(k_scale=cache["k_scale"][None], v_scale=cache["v_scale"][None])
        call(**pages, **scales)
        for name in scales:
            for bad in (None, scales[name][0], scales[name].int(), scales[name].cpu()):
                with pytest.raises(ValueError, match="k_scale|v_scale"):
                    call(**pages, **{**scales, name: bad})


def test_a_quantised_cache_on_the_cpu():
    from weight_streaming_expert_gb300 import PagedKVCache, copy_rows, read_cache
    cache = PagedKVCache(2, 4, 16, 3, 64, 64, dtype=E4M3, device="cpu")
    layer = cache.layer(1)
    assert set(layer) == {"k_cache", "v_cache", "k_scale", "v_scale"} and layer["k_scale"].shape == (4, 3, 16)
    assert set(PagedKVCache(1, 1, 16, 1, 64, 16, device="cpu").layer(0)) == {"k_cache", "v_cache"}
    with pytest.raises(ValueError, match="k_cache"):
        read_cache(**layer, slots=torch.zeros(1, dtype=torch.int64))
    with pytest.raises(ValueError, match="k_scale"):
        copy_rows(cache.k, cache.v, None, None, k_scale=cache.v_scale[0], v_scale=cache.v_scale)


def test_c_calls_refuse_before_the_gpu():
    import ctypes

    from weight_streaming_expert_gb300 import native as N
    L = N.lib()
    assert L.moe_qk_norm_rope_e4m3(None, None, None) == N.MOE_ERR_INVALID_ARG
    a = N.moe_qk_norm_rope_args_t(dtype=0, n_tokens=1, n_heads=0, n_kv_heads=1, head_dim=64, rotary_dim=0, eps=0.0, k=4096,
                                  v=4096, k_cache=4096, v_cache=4096, slots=4096, n_pages=1, page_size=16,
                                  k_page_stride=1024, k_row_stride=64, v_page_stride=1024, v_row_stride=64)
    s = N.moe_cache_scales_t()
    assert L.moe_qk_norm_rope_e4m3(ctypes.byref(a), ctypes.byref(s), None) == N.MOE_ERR_INVALID_ARG
    assert "scales" in N.last_error()
    s.k_scale = s.v_scale = 4096
    a.v_row_stride = 72
    assert L.moe_qk_norm_rope_e4m3(ctypes.byref(a), ctypes.byref(s), None) == N.MOE_ERR_INVALID_ARG
    assert "multiple of 16" in N.last_error()

    def read(**k):
        r = N.moe_read_e4m3_args_t(dtype=0, n=1, n_kv_heads=1, head_dim=64, k_cache=4096, v_cache=4096, k_page_stride=1024,
                                   k_row_stride=64, v_page_stride=1024, v_row_stride=64, scales=s, n_pages=1, page_size=16,
                                   slots=4096, k_out=4096, v_out=4096, k_token_stride=64, k_head_stride=64,
                                   v_token_stride=64, v_head_stride=64)
        for name, v in k.items():
            setattr(r, name, v)
        return L.moe_read_e4m3(ctypes.byref(r), None)

    assert L.moe_read_e4m3(None, None) == N.MOE_ERR_INVALID_ARG
    assert read(n=0) == N.MOE_OK and read(n_kv_heads=0) == N.MOE_OK
    for bad, text in ((dict(dtype=2), "dtype"), (dict(n=-1), "n and"), (dict(n_pages=0), "n_pages"), (dict(slots=None), "slots"),
                      (dict(slots=4100), "slots"), (dict(k_out=4104), "aligned"), (dict(k_row_stride=72), "16 bytes"),
                      (dict(v_head_stride=4), "8 elements"), (dict(scales=N.moe_cache_scales_t()), "scales")):
        assert read(**bad) == N.MOE_ERR_INVALID_ARG, bad
        assert text in N.last_error(), (bad, N.last_error())
    assert read(head_dim=96) == N.MOE_ERR_UNSUPPORTED
    args = [4096, 4096, 1, 64, 64, 64, 64, 16, 16, 1, 16, 1, 4096, 4096, 1, None]
    for at, bad, status in ((0, None, 1), (2, 0, 1), (9, 0, 1), (11, 0, 1), (12, None, 1), (13, 4100, 1), (14, -1, 1), (14, 65, 2)):
        assert L.moe_copy_scales(*(args[:at] + [bad] + args[at + 1:])) == status
    assert L.moe_copy_scales(*(args[:14] + [0, None])) == N.MOE_OK
