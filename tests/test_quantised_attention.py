"""Attention over the quantised cache (include/attention.h) against the formula
in 64 bits on what the codes stand for.

Tolerances, with h half a step of the element type, u = 2^-24, and for a row the
softmax probabilities pi_j, the scales 2^(e_j) and 2^(f_j) and the codes v_jd:
  * queries are exact in the products; a score of D terms, its two factors and
    the sum with f_j in fp32 are off by at most d = (D + 8) u scale sum |q k|
    plus u (|w| + |f|) where w is the score in powers of two, and taking the
    maximum off it adds u |w - M|: a relative error of the probability of 2 d +
    3 u W, W = max |w| + max |f|; the exponential itself and the running sums add
    at most (n + 64) u;
  * a probability times its value's scale is rounded once to fp16 against a
    largest one of at least 1 (per warp; the largest of a warp is at most that of
    all): a relative 2^-11, or the half step 2^-25 of that largest one;
  * the output is rounded once.
Chunks of more than 64 rows, and all rows over a shared prefix if they are more
than 64 together, go through 16 bits: their probabilities are rounded to the
element type, which the tolerance of test_attention counts (fp16 holds these
codes times their scales exactly)."""
import math

import pytest
import torch

from tests.test_attention import DEV, Case
from tests.test_quantised_cache import quantised

E4M3 = torch.float8_e4m3fn
U = 2.0 ** -24


class CodeCase(Case):
    """A Case whose keys and values are held as codes; the scales of rows that no
    position takes may be anything, and their codes NaN.  `spread`: keys and
    values are multiplied by powers of two up to 2^+-spread, row by row."""

    def __init__(self, *a, spread=0, **k):
        super().__init__(*a, **k)
        g = torch.Generator().manual_seed(77)
        self.codes, self.scales, self.exponents = {}, {}, {}
        for name in "kv":
            x = getattr(self, name).float()
            if spread and name == "v":
                x = x * torch.exp2(torch.randint(-spread, spread + 1, x.shape[:3], generator=g).float())[..., None]
            bytes_, e = quantised(x)
            empty = x.isnan().all(-1)
            scale = torch.where(empty, torch.randint(0, 256, e.shape, generator=g), e + 127).to(torch.uint8)
            self.codes[name], self.scales[name] = bytes_, scale.transpose(1, 2).contiguous()
        self.read_codes()

    def read_codes(self):
        """What the codes of each sequence stand for, and its values' scales."""
        self.ks, self.vs, self.fs = [], [], []
        for b, n in enumerate(self.kv_lens):
            n = max(0, n)
            pages = self.table[b, :-(-n // self.page)].long()
            row = {}
            for name in "kv":
                c = self.codes[name][pages].view(E4M3).double().flatten(0, 1)[:n]
                e = self.scales[name].transpose(1, 2)[pages].flatten(0, 1)[:n].double() - 127
                row[name] = torch.ldexp(c, e[..., None])
                row["e" + name] = e
            self.ks.append(row["k"])
            self.vs.append(row["v"])
            self.fs.append(row["ev"])

    def code_inputs(self):
        return dict(k_cache=self.codes["k"].to(DEV).view(E4M3), v_cache=self.codes["v"].to(DEV).view(E4M3),
                    k_scale=self.scales["k"].to(DEV), v_scale=self.scales["v"].to(DEV))

    def inputs(self):
        return {**super().inputs(), **self.code_inputs()}

    def sees(self, b):
        m, n = self.q_lens[b], max(0, self.kv_lens[b])
        i, j = torch.arange(m, device=DEV)[:, None], torch.arange(n, device=DEV)[None, :]
        if self.tree is None:
            return j <= n - m + i
        rows = self.tree[self.starts[b]:self.starts[b] + m]
        return torch.tensor([[c < n - m or (rows[r] >> (c - n + m)) & 1 for c in range(n)] for r in range(m)],
                            dtype=torch.bool, device=DEV).view(m, n)

    def check(self, out, lse, dtype, known_nan=None):
        h = torch.finfo(dtype).eps / 2
        chunks = max(self.q_lens + [0]) * self.group > 64 or (getattr(self, "prefix", 0) and
                                                              self.starts[-1] * self.group > 64)
        assert out.dtype == dtype
        for b, m in enumerate(self.q_lens):
            n, rows = max(0, self.kv_lens[b]), slice(self.starts[b], self.starts[b + 1])
            sees = self.sees(b)
            none = ~sees.any(1)
            for hq in range(self.Hq):
                q = self.q[rows, hq].to(DEV).double()
                k, v = (x[:, hq // self.group].to(DEV) for x in (self.ks[b], self.vs[b]))
                f = self.fs[b][:, hq // self.group].to(DEV)
                raw = q @ k.T * self.scale
                x = raw.masked_fill(~sees, -math.inf)
                top = x.amax(1, keepdim=True) if n else torch.full((m, 1), -math.inf, device=DEV, dtype=torch.double)
                top = torch.where(top == -math.inf, torch.zeros_like(top), top)
                p = torch.exp(x - top)
                total = p.sum(1, keepdim=True)
                want_lse = (total.log() + top)[:, 0]
                p = p / torch.where(total == 0, torch.ones_like(total), total)
                want = p @ v
                size = p @ v.abs()
                if n and m:
                    d = (self.D + 8) * U * self.scale * (q.abs() @ k.abs().T).amax(1, keepdim=True)
                    W = 1.45 * raw.abs().amax(1, keepdim=True) + f.abs().max()
                    soft = 2 * d + 3 * U * W + (n + 64) * U
                    floor = 2.0 ** -25 * (p * torch.exp2(f)).amax(1, keepdim=True) * torch.exp2(-f)[None] @ v.abs()
                else:
                    soft, floor = torch.zeros(m, 1, device=DEV), 0.0
                rounding = h if chunks else 2.0 ** -11
                tol = size * (rounding + soft) * 1.01 + floor + h * want.abs()
                if dtype == torch.float16:
                    tol = tol + 2.0 ** -25 * ((sees.double() @ v.abs()) / total.clamp_min(1) + 1 if chunks else 1)
                got = out[rows, hq].double()
                off = (got - want).abs() - tol
                assert (off <= 0).all(), f"seq {b} head {hq}: {off.max().item():.3g} past the bound"
                got_lse = lse[rows, hq].double()
                assert (got_lse[none] == -math.inf).all() and (got[none] == 0).all()
                lse_tol = (soft + 8 * U * (1 + want_lse.abs() + (f.abs().max() if n else 0))[:, None])[:, 0]
                assert ((got_lse - want_lse).abs() <= lse_tol)[~none].all()


def run(case, **more):
    from weight_streaming_expert_gb300 import PagedAttention
    attn = PagedAttention(case.Hq, case.Hk, case.D, device=DEV)
    x = case.inputs()
    x.update(more)
    out, lse = attn(return_lse=True, **x)
    assert attn.status() == 0
    case.check(out, lse, case.q.dtype)
    attn.close()
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("D", [64, 128])
def test_types_pages_and_dims(dtype, page, D):
    run(CodeCase([1, 5, 16], [77, 300, 40], 8, 2, D, page, dtype, seed=page + D))


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (2, 1), (5, 1), (8, 8), (20, 4), (14, 2), (48, 1), (64, 4), (64, 1), (100, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_head_layouts(Hq, Hk, D):
    run(CodeCase([3, 1], [200, 129], Hq, Hk, D, 64, seed=Hq))


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 63, 64, 65, 111, 112, 113, 127, 128, 129, 255, 256, 257, 1023, 1025])
def test_lengths_of_one_token(n):
    run(CodeCase([1], [n], 4, 1, 128, 16, seed=n))
    run(CodeCase([1], [n], 4, 1, 64, 16, "fp16", seed=n))


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 17, 31, 32, 33, 64, 100, 257])
@pytest.mark.parametrize("before", [0, 1, 130])
def test_chunk_lengths(m, before):
    run(CodeCase([m], [m + before], 4, 2, 64, 32, "fp16", seed=m))
    run(CodeCase([m], [m + before], 2, 1, 128, 32, "bf16", seed=m))


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hk,ms", [(8, 2, [1, 1, 4, 2]), (5, 1, [6, 2, 1, 12]), (16, 1, [4, 1, 3]), (3, 3, [21, 2])])
def test_ragged_batches_and_empty_sequences(Hq, Hk, ms):
    q_lens = [0] + ms + [0]
    kv_lens = [0] + [m + 37 * i * i for i, m in enumerate(ms)] + [55]
    run(CodeCase(q_lens, kv_lens, Hq, Hk, 128, 16, seed=Hq))
    run(CodeCase(q_lens, kv_lens, Hq, Hk, 64, 64, "fp16", seed=Hq))


@pytest.mark.gpu
@pytest.mark.parametrize("n", [5, 13, 32, 64])
@pytest.mark.parametrize("D", [64, 128])
def test_trees(n, D):
    import random
    rng, tree = random.Random(n), []
    for _ in range(3):
        seen = []
        for i in range(n):
            parent = rng.randrange(-1, i) if i else -1
            seen.append((seen[parent] if parent >= 0 else 0) | 1 << i)
        tree += seen
    tree[1] = 0  # sees only what is before the chunk
    run(CodeCase([n] * 3, [n, n + 100, n + 777], 2, 2, D, 16, tree=tree, seed=n))


@pytest.mark.gpu
def test_long_sequences_are_cut_and_joined():
    run(CodeCase([1, 6, 1], [20000, 9999, 130], 20, 4, 128, 64, seed=1))
    run(CodeCase([1] * 40, [100 + 371 * i for i in range(40)], 8, 2, 64, 16, "fp16", seed=2))
    run(CodeCase([1] * 700, [1 + i % 300 for i in range(700)], 4, 1, 128, 16, seed=3))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128])
def test_scales_far_apart(dtype, D):
    """Values of one head between 2^-20 and 2^20: each counts with its probability."""
    run(CodeCase([4, 1], [600, 333], 6, 2, D, 32, "bf16", seed=9, spread=20) if dtype == "bf16" else
        CodeCase([4, 1], [600, 333], 6, 2, D, 32, "fp16", seed=9, spread=5))


@pytest.mark.gpu
def test_peaked_and_flat_scores():
    run(CodeCase([2], [3000], 4, 1, 128, 64, seed=4, scale=3.0))
    run(CodeCase([2], [3000], 4, 1, 128, 64, "fp16", seed=5, scale=1e-6))


@pytest.mark.gpu
@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** -20, 2.0 ** 30, 2.0 ** 90])
def test_queries_of_any_size(size):
    """A power of two of the queries and its inverse in the scale change nothing."""
    case = CodeCase([3, 1], [200, 90], 5, 1, 128, 16, seed=6)
    want = run(case)
    case.q = (case.q.double() * size).bfloat16()
    case.scale = case.scale / size
    assert torch.equal(run(case), want)


@pytest.mark.gpu
@pytest.mark.parametrize("D,m,Hq", [(64, 6, 4), (128, 6, 4), (128, 3, 20), (128, 40, 4)])
def test_hidden_codes_may_be_anything_and_seen_nan_show(D, m, Hq):
    """NaN codes in rows of the chunk that only later tokens see, and in seen ones."""
    from weight_streaming_expert_gb300 import PagedAttention
    case = CodeCase([m, 2], [m + 50, 300], Hq, 2, D, 16, seed=8)
    attn = PagedAttention(Hq, 2, D, device=DEV)
    clean = case.inputs()
    want, want_lse = attn(return_lse=True, **clean)
    slot = lambda b, pos: (int(case.table[b, pos // 16]), pos % 16)
    page, row = slot(0, 50 + m - 1)  # the last token of the chunk: hidden from the others
    case.codes["v"][page, row, 1, 5] = 0x7f
    case.codes["v"][page, row, 0, D - 1] = 0xff
    x = case.inputs()
    out, lse = attn(return_lse=True, **x)
    assert torch.equal(out[:m - 1], want[:m - 1]) and torch.equal(out[m:], want[m:]) and torch.equal(lse, want_lse)
    group = Hq // 2
    bad = torch.zeros(Hq, D, dtype=torch.bool, device=DEV)
    bad[group:, 5] = True
    bad[:group, D - 1] = True
    assert torch.equal(out[m - 1].isnan(), bad) and torch.equal(out[m - 1][~bad], want[m - 1][~bad])
    case.codes["k"][page, row] = 0x7f  # a key: the rows that see it are NaN throughout
    x = case.inputs()
    out, lse = attn(return_lse=True, **x)
    assert torch.equal(out[:m - 1], want[:m - 1]) and out[m - 1].isnan().all() and lse[m - 1].isnan().all()
    page, row = slot(1, 17)  # seen by all of its sequence
    case.codes["v"][page, row, 0, 3] = 0x7f
    out = attn(**case.inputs())
    assert out[m:, :group, 3].isnan().all() and not out[m:, group:].isnan().any()
    assert not out[m:, :group, 4:].isnan().any()
    attn.close()


@pytest.mark.gpu
def test_unused_rows_stay_as_they_were_and_strides():
    from weight_streaming_expert_gb300 import PagedAttention
    case = CodeCase([2, 1], [70, 33], 4, 2, 128, 16, seed=10)
    x = case.inputs()
    wide = torch.full((5, 6, 160), 7.0, device=DEV).bfloat16()
    q = torch.zeros(5, 9, 128, device=DEV).bfloat16()
    q[:3, 2:6] = x["q"]
    pool = {}
    for n in "kv":
        codes = torch.full((x[n + "_cache"].shape[0], 20, 2, 128), 0x7f, dtype=torch.uint8, device=DEV)
        codes[:, :16] = x[n + "_cache"].view(torch.uint8)
        pool[n + "_cache"] = codes[:, :16].view(E4M3)
        scale = torch.full((codes.shape[0], 3, 32), 255, dtype=torch.uint8, device=DEV)
        scale[:, :2, :16] = x[n + "_scale"]
        pool[n + "_scale"] = scale[:, :2, :16]
    attn = PagedAttention(4, 2, 128, device=DEV)
    out = wide[:, 1:5, :128]
    got, lse = attn(**{**x, **pool, "q": q[:, 2:6], "out": out, "return_lse": True})
    case.check(out, lse, torch.bfloat16)
    assert (wide[3:] == 7).all() and (wide[:, 0] == 7).all() and (wide[:, :, 128:] == 7).all()
    attn.close()


@pytest.mark.gpu
@pytest.mark.parametrize("m,Hq", [(1, 4), (3, 20), (90, 4)])
def test_captured_with_changing_lengths_and_streams(m, Hq):
    from weight_streaming_expert_gb300 import PagedAttention
    case = CodeCase([m, m], [m + 400, m + 30], Hq, 2, 128, 16, seed=11)
    attn = PagedAttention(Hq, 2, 128, device=DEV)
    x = case.inputs()
    want = attn(**x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = attn(**x, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = attn(**x, return_lse=True)
    x["kv_lens"].copy_(torch.tensor([m + 111, m + 29]))
    case.kv_lens = [m + 111, m + 29]
    case.read_codes()
    graph.replay()
    torch.cuda.synchronize()
    case.check(out, lse, torch.bfloat16)
    assert attn.status() == 0
    attn.close()


@pytest.mark.gpu
def test_one_handle_over_codes_and_16_bits_in_turn():
    """A call leaves nothing behind for one of another kind, and the same call gives the same bits."""
    from tests.test_attention import Case as Plain
    from weight_streaming_expert_gb300 import PagedAttention
    attn = PagedAttention(8, 2, 128, device=DEV)
    calls = [CodeCase([1] * 3, [900, 50, 333], 8, 2, 128, 16, seed=1), Plain([1] * 3, [900, 50, 333], 8, 2, 128, 16, seed=2),
             CodeCase([40, 2], [300, 99], 8, 2, 128, 32, seed=3), Plain([40, 2], [300, 99], 8, 2, 128, 64, seed=4),
             CodeCase([6], [5000], 8, 2, 128, 64, seed=5)]
    first = [attn(**c.inputs()) for c in calls]
    for _ in range(3):
        for c, want in zip(calls, first):
            assert torch.equal(attn(**c.inputs()), want)
    assert attn.status() == 0
    attn.close()


@pytest.mark.gpu
def test_chunks_in_turns_with_a_small_workspace():
    """Sequences that do not fit the workspace together take turns."""
    import ctypes

    from weight_streaming_expert_gb300 import native as N
    case = CodeCase([40, 90, 3], [300, 90, 77], 4, 2, 64, 16, seed=12)
    x = case.inputs()
    out = torch.empty_like(x["q"])
    lse = torch.empty(x["q"].shape[:2], device=DEV)
    L = N.lib()
    h = L.moe_attn_create(4, 2, 64)
    k, v = x["k_cache"], x["v_cache"]
    a = N.moe_attn_args_t(dtype=0, batch=3, n_tokens=133, max_q_len=90, scale=case.scale, q=x["q"].data_ptr(),
                          q_token_stride=256, q_head_stride=64, k_cache=k.data_ptr(), v_cache=v.data_ptr(),
                          k_page_stride=k.stride(0), k_row_stride=k.stride(1), v_page_stride=v.stride(0),
                          v_row_stride=v.stride(1), n_pages=k.shape[0], page_size=16, block_table=x["block_table"].data_ptr(),
                          table_stride=x["block_table"].shape[1], q_starts=x["q_starts"].data_ptr(),
                          kv_lens=x["kv_lens"].data_ptr(), out=out.data_ptr(), out_token_stride=256, out_head_stride=64,
                          lse=lse.data_ptr())
    ks, vs = x["k_scale"], x["v_scale"]
    s = N.moe_cache_scales_t(ks.data_ptr(), vs.data_ptr(), ks.stride(0), ks.stride(1), vs.stride(0), vs.stride(1))
    o = N.moe_attn_opts_t(ctypes.pointer(s), 0, None, 0)
    need = L.moe_attn_workspace(h, ctypes.byref(a), ctypes.byref(o))
    assert need == 3 * x["block_table"].shape[1] * (16 * 2 * 64 * 4 + 16)
    room = torch.zeros(need + 16, dtype=torch.uint8, device=DEV)
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    for size in (need, need // 3 * 2 + 5, need // 3):
        o.workspace, o.workspace_bytes = room.data_ptr(), size
        room.fill_(0xff)
        out.zero_()
        assert L.moe_attn_forward_ex(h, ctypes.byref(a), ctypes.byref(o), stream) == 0, N.last_error()
        assert L.moe_attn_get_status(h) == 0
        case.check(out, lse, torch.bfloat16)
        assert (room[size:] == 0xff).all()
    o.workspace_bytes = need // 3 - 1
    assert L.moe_attn_forward_ex(h, ctypes.byref(a), ctypes.byref(o), stream) == N.MOE_ERR_INVALID_ARG
    assert "workspace" in N.last_error()
    L.moe_attn_destroy(h)


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 3, 50])
def test_bad_pages_and_lengths_are_reported(m):
    from weight_streaming_expert_gb300 import PagedAttention
    from weight_streaming_expert_gb300 import native as N
    case = CodeCase([m, m], [m + 60, m + 40], 4, 2, 64, 16, seed=13)
    attn = PagedAttention(4, 2, 64, device=DEV)
    x = case.inputs()
    want = attn(**x)
    table = x["block_table"].clone()
    table[0, 1] = 1 << 20
    out = attn(**{**x, "block_table": table})
    assert attn.status() == N.MOE_ERR_INVALID_ARG and attn.status() == 0
    assert torch.equal(out[m:], want[m:]) and not out.isnan().any()
    x["kv_lens"][0] = 1 << 20
    attn(**x)
    assert attn.status() == N.MOE_ERR_INVALID_ARG
    attn.close()


@pytest.mark.gpu
def test_refusals():
    from weight_streaming_expert_gb300 import PagedAttention
    case = CodeCase([2], [40], 4, 2, 64, 16)
    attn = PagedAttention(4, 2, 64, device=DEV)
    good = case.inputs()
    attn(**good)
    for name in ("k_cache", "v_cache"):
        for bad in (good[name].view(torch.uint8), good[name].float().bfloat16(), None):
            with pytest.raises(ValueError, match="k_cache|v_cache"):
                attn(**{**good, name: bad})
    for name in ("k_scale", "v_scale"):
        t = good[name]
        for bad in (None, t.int(), t[:, :1], t.cpu(), t.transpose(1, 2), 4):
            with pytest.raises(ValueError, match="k_scale|v_scale"):
                attn(**{**good, name: bad})
    odd = torch.zeros(t.shape[0], 2, 24, dtype=torch.uint8, device=DEV)[:, :, :16]
    from weight_streaming_expert_gb300.native import MoEError
    with pytest.raises(MoEError, match="multiple of 16"):
        attn(**{**good, "k_scale": odd})
    attn.close()
