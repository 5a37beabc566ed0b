"""Attention of a batch whose sequences begin with the same pages (prefix_len)
against the formula in 64 bits over the whole sequences.

Tolerances: those of test_attention (16-bit caches) and of
test_quantised_attention.  A token's two results are joined in fp32 from their
unnormalised sums: two factors, products and a sum more, which the 64 u beside
the n u of a sum's terms hold."""
import math
import random
import struct

import pytest
import torch

from tests.test_attention import DEV, TYPES, Case
from tests.test_quantised_attention import CodeCase, quantised


class Shared(Case):
    """`own`: positions of each sequence after the prefix, the new tokens
    included.  Pages lie anywhere; unused rows hold NaN; the other rows of the
    table name no pages for the prefix."""

    def __init__(self, q_lens, own, prefix, Hq, Hk, D, page, dtype="bf16", seed=0, tree=None, codes=False, scale=None):
        g = torch.Generator().manual_seed(seed)
        dt = TYPES[dtype]
        self.q_lens, self.own, self.prefix, self.D, self.page = q_lens, own, prefix, D, page
        self.kv_lens = [prefix + n for n in own]
        self.Hq, self.Hk, self.group = Hq, Hk, Hq // Hk
        self.tree, self.scale = tree, D ** -0.5 if scale is None else scale
        first = prefix // page
        need = [-(-n // page) for n in own]
        total, width = first + sum(need) + 3, first + max(need + [1])
        order = torch.randperm(total, generator=g).to(torch.int32)
        self.full = torch.full((len(q_lens), width), -1, dtype=torch.int32)  # with the prefix in every row
        self.full[:, :first] = order[:first]
        at = first
        for b, n in enumerate(need):
            self.full[b, first:first + n] = order[at:at + n]
            at += n
        self.table = self.full
        self.k, self.v = (torch.full((total, page, Hk, D), math.nan, dtype=dt) for _ in range(2))
        for b, n in enumerate(self.kv_lens):
            for j in range(0 if b == 0 else first, -(-n // page)):
                p, m = int(self.full[b, j]), min(page, n - j * page)
                for t in (self.k, self.v):
                    t[p, :m] = torch.randn(m, Hk, D, generator=g).to(dt)
        self.starts = [0]
        for n in q_lens:
            self.starts.append(self.starts[-1] + n)
        self.q = torch.randn(self.starts[-1], Hq, D, generator=g).to(dt)
        self.ks, self.vs = [], []
        for b, n in enumerate(self.kv_lens):
            pages = self.full[b, :-(-n // page)].long()
            self.ks.append(self.k[pages].flatten(0, 1)[:n])
            self.vs.append(self.v[pages].flatten(0, 1)[:n])
        if codes:
            self.codes, self.scales = {}, {}
            for name in "kv":
                x = getattr(self, name).float()
                bytes_, e = quantised(x)
                scale_ = torch.where(x.isnan().all(-1), torch.randint(0, 256, e.shape, generator=g), e + 127)
                self.codes[name], self.scales[name] = bytes_, scale_.to(torch.uint8).transpose(1, 2).contiguous()
            CodeCase.read_codes(self)
        self.with_codes = codes

    def inputs(self):
        x = Case.inputs(self)
        if self.with_codes:
            x.update(CodeCase.code_inputs(self))
        table = self.full.clone()
        table[1:, :self.prefix // self.page] = 1 << 30  # not read
        x.update(block_table=table.to(DEV), prefix_len=self.prefix)
        return x

    def check(self, out, lse, dtype):
        if self.with_codes:
            CodeCase.check(self, out, lse, dtype)
        else:
            Case.check(self, out, lse, dtype)

    def sees(self, b):
        return CodeCase.sees(self, b)


def run(case, **more):
    from weight_streaming_expert_gb300 import PagedAttention
    attn = PagedAttention(case.Hq, case.Hk, case.D, device=DEV)
    x = case.inputs()
    x.update(more)
    out, lse = attn(return_lse=True, **x)
    assert attn.status() == 0
    case.check(out, lse, case.q.dtype)
    again = attn(**x)
    assert torch.equal(again, out)
    attn.close()
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("page,prefix", [(16, 16), (16, 240), (32, 640), (64, 64), (128, 1280), (256, 256)])
@pytest.mark.parametrize("D", [64, 128])
def test_types_pages_and_dims(codes, dtype, page, prefix, D):
    run(Shared([1, 3, 2], [1, 70, 300], prefix, 8, 2, D, page, dtype, seed=page + D, codes=codes))


@pytest.mark.gpu
@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (5, 1), (8, 8), (20, 4), (14, 2), (64, 1), (128, 1), (128, 2)])
def test_head_layouts(codes, Hq, Hk):
    run(Shared([1, 2, 1, 1], [5, 130, 1, 64], 208, Hq, Hk, 128, 16, seed=Hq, codes=codes))


@pytest.mark.gpu
@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("batch", [1, 2, 15, 16, 17, 33, 64, 129, 300])
def test_batches_of_single_tokens(codes, batch):
    rng = random.Random(batch)
    run(Shared([1] * batch, [rng.randint(1, 200) for _ in range(batch)], 512, 8, 1, 64, 16, "fp16", seed=batch, codes=codes))


@pytest.mark.gpu
@pytest.mark.parametrize("codes", [False, True])
def test_the_largest_batch(codes):
    rng = random.Random(9)
    run(Shared([1] * 4096, [rng.randint(1, 20) for _ in range(4096)], 32, 1, 1, 64, 16, seed=9, codes=codes))


@pytest.mark.gpu
@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("m", [1, 7, 16, 31, 33, 64, 65, 100, 260])
def test_chunks(codes, m):
    run(Shared([m, m // 2, 0, 1], [m, m + 5, 40, 1], 320, 4, 2, 128, 32, seed=m, codes=codes))


@pytest.mark.gpu
@pytest.mark.parametrize("codes", [False, True])
def test_long_prefixes_are_cut_and_joined(codes):
    run(Shared([1] * 8, [300 - 37 * i for i in range(8)], 20000 // 64 * 64, 20, 4, 128, 64, seed=1, codes=codes))
    run(Shared([4] * 3, [4000, 900, 2500], 2048, 16, 2, 64, 128, "fp16", seed=2, codes=codes))


@pytest.mark.gpu
@pytest.mark.parametrize("codes", [False, True])
def test_many_tokens_whose_prefix_runs_by_itself(codes):
    rng = random.Random(5)
    run(Shared([1] * 260, [rng.randint(1, 100) for _ in range(260)], 3200, 32, 4, 128, 64, seed=5, codes=codes))
    run(Shared([rng.randint(0, 5) for _ in range(90)], [rng.randint(5, 300) for _ in range(90)], 176, 24, 2, 64, 16, "fp16",
               seed=6, codes=codes))


@pytest.mark.gpu
def test_chunks_over_codes_in_turns():
    """With room for one sequence's pages the prefix is unpacked once and the sequences take turns."""
    import ctypes

    from weight_streaming_expert_gb300 import native as N
    case = Shared([30, 70, 2], [90, 70, 33], 96, 6, 2, 64, 16, seed=12, codes=True)
    x = case.inputs()
    out, lse = torch.empty_like(x["q"]), torch.empty(x["q"].shape[:2], device=DEV)
    L = N.lib()
    h = L.moe_attn_create(6, 2, 64)
    k, v, ks, vs, table = (x[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale", "block_table"))
    a = N.moe_attn_args_t(dtype=0, batch=3, n_tokens=102, max_q_len=70, scale=case.scale, q=x["q"].data_ptr(),
                          q_token_stride=384, q_head_stride=64, k_cache=k.data_ptr(), v_cache=v.data_ptr(),
                          k_page_stride=k.stride(0), k_row_stride=k.stride(1), v_page_stride=v.stride(0),
                          v_row_stride=v.stride(1), n_pages=k.shape[0], page_size=16, block_table=table.data_ptr(),
                          table_stride=table.shape[1], q_starts=x["q_starts"].data_ptr(), kv_lens=x["kv_lens"].data_ptr(),
                          out=out.data_ptr(), out_token_stride=384, out_head_stride=64, lse=lse.data_ptr())
    s = N.moe_cache_scales_t(ks.data_ptr(), vs.data_ptr(), ks.stride(0), ks.stride(1), vs.stride(0), vs.stride(1))
    o = N.moe_attn_opts_t(ctypes.pointer(s), 96, None, 0)
    wanted = L.moe_attn_workspace(h, ctypes.byref(a), ctypes.byref(o))
    one = (table.shape[1] - 6) * 16 * 2 * 64 * 4 + table.shape[1] * 16
    room = torch.zeros(wanted + 16, dtype=torch.uint8, device=DEV)
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    for size in (wanted, wanted - one, wanted - 2 * one):
        o.workspace, o.workspace_bytes = room.data_ptr(), size
        room.fill_(0xff)
        out.zero_()
        assert L.moe_attn_forward_ex(h, ctypes.byref(a), ctypes.byref(o), stream) == 0, N.last_error()
        assert L.moe_attn_get_status(h) == 0
        case.check(out, lse, torch.bfloat16)
        assert (room[size:] == 0xff).all()
    o.workspace_bytes = wanted - 2 * one - 1
    assert L.moe_attn_forward_ex(h, ctypes.byref(a), ctypes.byref(o), stream) == N.MOE_ERR_INVALID_ARG
    L.moe_attn_destroy(h)


@pytest.mark.gpu
@pytest.mark.parametrize("codes", [False, True])
def test_starts_that_make_no_sense_are_reported(codes):
    from weight_streaming_expert_gb300 import PagedAttention
    from weight_streaming_expert_gb300 import native as N
    case = Shared([3, 2, 4], [40, 30, 9], 64, 4, 2, 64, 16, seed=14, codes=codes)
    attn = PagedAttention(4, 2, 64, device=DEV)
    x = case.inputs()
    attn(**x)
    for starts in ([5, 9, 3, 3], [0, 9, 2, 4], [-7, 3, 5, 1 << 30], [9, 6, 3, 0], [1 << 30, 0, 1, 2]):
        out = attn(**{**x, "q_starts": torch.tensor(starts, dtype=torch.int32, device=DEV)})
        assert attn.status() == N.MOE_ERR_INVALID_ARG and out.shape == x["q"].shape
    attn.close()


@pytest.mark.gpu
@pytest.mark.parametrize("codes", [False, True])
def test_trees_after_a_prefix(codes):
    rng, tree, n = random.Random(3), [], 13
    for _ in range(4):
        seen = []
        for i in range(n):
            parent = rng.randrange(-1, i) if i else -1
            seen.append((seen[parent] if parent >= 0 else 0) | 1 << i)
        tree += seen
    tree[5] = 0  # the prefix and what is before the chunk
    run(Shared([n] * 4, [n, n + 1, n + 200, n + 40], 96, 4, 2, 64, 16, "fp16", tree=tree, seed=3, codes=codes))


@pytest.mark.gpu
@pytest.mark.parametrize("codes", [False, True])
def test_the_same_as_without(codes):
    """Up to rounding, what the same sequences give as separate ones."""
    from weight_streaming_expert_gb300 import PagedAttention
    case = Shared([1, 2, 3], [9, 80, 33], 448, 8, 2, 128, 64, seed=4, codes=codes)
    attn = PagedAttention(8, 2, 128, device=DEV)
    x = case.inputs()
    shared = attn(**x)
    x.update(block_table=case.full.to(DEV), prefix_len=0)
    assert (attn(**x).float() - shared.float()).abs().max() < 0.02
    attn.close()


@pytest.mark.gpu
@pytest.mark.parametrize("codes", [False, True])
def test_nan_that_is_seen_shows_and_hidden_does_not(codes):
    from weight_streaming_expert_gb300 import PagedAttention
    case = Shared([3, 1], [40, 7], 160, 4, 2, 64, 16, seed=5, codes=codes)
    attn = PagedAttention(4, 2, 64, device=DEV)
    want = attn(**case.inputs())

    def poison(b, pos):
        page, row = int(case.full[b, pos // 16]), pos % 16
        if codes:
            case.codes["v"][page, row, 1, 7] = 0x7f
        else:
            case.v[page, row, 1, 7] = math.nan

    poison(0, 160 + 39)  # the last token of sequence 0
    out = attn(**case.inputs())
    bad = out.isnan()
    assert bad[2, 2:, 7].all() and bad.sum() == 2
    assert torch.equal(out[~bad], want[~bad])
    poison(1, 100)  # of the prefix is another page than sequence 0's only in the oracle's eyes
    page = int(case.full[0, 6])
    assert page == int(case.full[1, 6])
    out = attn(**case.inputs())
    assert out[:, 2:, 7].isnan().all() and not out[:, :2].isnan().any()
    attn.close()


@pytest.mark.gpu
@pytest.mark.parametrize("codes", [False, True])
def test_captured_with_changing_lengths_and_shared_workspaces(codes):
    """Two captured calls of one handle, replayed in turn; their workspaces come from the graphs' pool."""
    from weight_streaming_expert_gb300 import PagedAttention
    attn = PagedAttention(8, 2, 64, device=DEV)
    cases = [Shared([1] * 4, [100, 30, 1, 64], 256, 8, 2, 64, 32, seed=6, codes=codes),
             Shared([5, 2], [33, 700], 1024, 8, 2, 64, 32, seed=7, codes=codes)]
    graphs, pool = [], None
    for c in cases:
        x = c.inputs()
        attn(**x)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=pool):
            out, lse = attn(**x, return_lse=True)
        pool = graph.pool()
        graphs.append((graph, x, out, lse))
    for turn in range(3):
        for c, (graph, x, out, lse) in zip(cases, graphs):
            graph.replay()
            torch.cuda.synchronize()
            c.check(out, lse, torch.bfloat16)
    c, (graph, x, out, lse) = cases[0], graphs[0]
    c.own, c.kv_lens = [90, 30, 1, 50], [346, 286, 257, 306]
    c.ks, c.vs = [k[:n] for k, n in zip(c.ks, c.kv_lens)], [v[:n] for v, n in zip(c.vs, c.kv_lens)]
    if codes:
        c.fs = [f[:n] for f, n in zip(c.fs, c.kv_lens)]
    x["kv_lens"].copy_(torch.tensor(c.kv_lens))
    graph.replay()
    torch.cuda.synchronize()
    c.check(out, lse, torch.bfloat16)
    assert attn.status() == 0
    attn.close()


@pytest.mark.gpu
@pytest.mark.parametrize("codes", [False, True])
def test_on_another_stream_and_rows_behind_the_last_sequence(codes):
    from weight_streaming_expert_gb300 import PagedAttention
    case = Shared([1, 2], [20, 30], 64, 4, 2, 128, 16, seed=8, codes=codes)
    attn = PagedAttention(4, 2, 128, device=DEV)
    x = case.inputs()
    q = torch.cat((x["q"], torch.full((4, 4, 128), math.nan, device=DEV).bfloat16()))
    out = torch.full((7, 4, 128), 5.0, device=DEV).bfloat16()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, lse = attn(**{**x, "q": q, "out": out}, return_lse=True, stream=side)
    side.synchronize()
    assert (out[3:] == 5).all() and attn.status() == 0
    case.check(out[:3], lse[:3], torch.bfloat16)
    attn.close()


@pytest.mark.gpu
@pytest.mark.parametrize("codes", [False, True])
def test_sequences_shorter_than_the_prefix_and_bad_pages_are_reported(codes):
    from weight_streaming_expert_gb300 import PagedAttention
    from weight_streaming_expert_gb300 import native as N
    case = Shared([1, 1, 1], [20, 30, 9], 64, 4, 2, 64, 16, seed=9, codes=codes)
    attn = PagedAttention(4, 2, 64, device=DEV)
    x = case.inputs()
    want = attn(**x)
    for length in (64, 63, 0, -5, 1 << 30):
        kv = x["kv_lens"].clone()
        kv[1] = length
        out = attn(**{**x, "kv_lens": kv})
        assert attn.status() == N.MOE_ERR_INVALID_ARG
        if length < 1 << 30:  # else cut to the table, whose rows hold NaN there; other shares, other roundings
            assert torch.equal(out[[0, 2]], want[[0, 2]]) and not out.isnan().any()
        assert not out[[0, 2]].isnan().any()
    table = x["block_table"].clone()
    table[0, 1] = -7
    attn(**{**x, "block_table": table})
    assert attn.status() == N.MOE_ERR_INVALID_ARG and attn.status() == 0
    attn.close()


@pytest.mark.gpu
def test_refusals():
    from weight_streaming_expert_gb300 import PagedAttention
    from weight_streaming_expert_gb300.native import MoEError
    case = Shared([1, 1], [20, 30], 64, 4, 2, 64, 16)
    attn = PagedAttention(4, 2, 64, device=DEV)
    x = case.inputs()
    for bad, error in ((-16, ValueError), (16.0, ValueError), (None, ValueError), (1 << 31, ValueError), (24, MoEError),
                       (1 << 20, MoEError)):
        with pytest.raises(error, match="prefix_len"):
            attn(**{**x, "prefix_len": bad})
    attn.close()


@pytest.mark.gpu
def test_nothing_to_do():
    from weight_streaming_expert_gb300 import PagedAttention
    case = Shared([1, 1], [20, 30], 64, 4, 2, 64, 16)
    attn = PagedAttention(4, 2, 64, device=DEV)
    x = case.inputs()
    x.update(q=x["q"][:0], q_starts=torch.zeros(3, dtype=torch.int32, device=DEV))
    assert attn(**x).shape == (0, 4, 64) and attn.status() == 0
    x = case.inputs()
    x.update(q_starts=torch.zeros(3, dtype=torch.int32, device=DEV), out=torch.full_like(x["q"], 3.0))
    assert (attn(**x) == 3).all() and attn.status() == 0
    attn.close()


def test_what_forks_share():
    from weight_streaming_expert_gb300 import PagedKVCache
    cache = PagedKVCache(1, 20, 16, 1, 64, 320, device="cpu")
    extend = lambda s, n: cache.table.extend(s, n)
    a = cache.open()
    extend(a, 40)
    b = cache.fork(a)
    assert cache.shared_prefix([a, b]) == 32 and cache.shared_prefix([a]) == 32
    assert cache.shared_prefix([a, b], new=9) == 16 and cache.shared_prefix([a, b], new=100) == 0
    extend(a, 1)
    extend(b, 30)
    assert cache.shared_prefix([a, b]) == 32
    c = cache.open()
    extend(c, 5)
    assert cache.shared_prefix([a, b, c]) == 0 and cache.shared_prefix([]) == 0
    cache.truncate(a, 32)
    assert cache.shared_prefix([a, b]) == 16  # its last position is the new token's


def test_c_call_refuses_before_the_gpu():
    import ctypes

    from weight_streaming_expert_gb300 import native as N
    L = N.lib()
    fake = ctypes.create_string_buffer(struct.pack("3i", 4, 2, 64), 4096)  # a handle's first numbers

    def call(prefix=16, scales=None, workspace=4096, size=1 << 40, **k):
        a = N.moe_attn_args_t(dtype=0, batch=1, n_tokens=1, max_q_len=1, scale=1.0, q=4096, q_token_stride=256,
                              q_head_stride=64, k_cache=4096, v_cache=4096, k_page_stride=2048, k_row_stride=128,
                              v_page_stride=2048, v_row_stride=128, n_pages=4, page_size=16, block_table=4096,
                              table_stride=4, q_starts=4096, kv_lens=4096, out=4096, out_token_stride=256,
                              out_head_stride=64)
        for name, v in k.items():
            setattr(a, name, v)
        o = N.moe_attn_opts_t(ctypes.pointer(scales) if scales else None, prefix, workspace, size)
        return L.moe_attn_forward_ex(fake, ctypes.byref(a), ctypes.byref(o), None)

    good = N.moe_cache_scales_t(4096, 4096, 64, 32, 64, 32)
    for bad, text in ((dict(prefix=-16), "prefix_len"), (dict(prefix=8), "whole pages"), (dict(prefix=80), "4 pages"),
                      (dict(workspace=None), "workspace"), (dict(workspace=4104), "workspace"), (dict(size=100), "workspace"),
                      (dict(scales=N.moe_cache_scales_t()), "scales"),
                      (dict(scales=N.moe_cache_scales_t(4096, 4104, 64, 32, 64, 32)), "scales"),
                      (dict(scales=N.moe_cache_scales_t(4096, 4096, 64, 8, 64, 32)), "multiple of 16"),
                      (dict(scales=good, k_row_stride=136), "multiple of 16"), (dict(dtype=3), "dtype")):
        assert call(**bad) == N.MOE_ERR_INVALID_ARG, bad
        assert text in N.last_error(), (bad, N.last_error())
    assert call(batch=0) == N.MOE_OK and call(n_tokens=0, scales=good) == N.MOE_OK
    assert call(page_size=256, prefix=256, table_stride=1 << 20, n_tokens=1 << 30, max_q_len=1 << 30,
                size=1 << 62) == N.MOE_ERR_UNSUPPORTED
    assert "too much work" in N.last_error()
    assert L.moe_attn_workspace(None, None, None) == 0
