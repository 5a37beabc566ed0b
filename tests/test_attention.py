"""Attention of new tokens over the paged cache (include/attention.h) against
the formula in 64 bits, sequence by sequence and head by head.

Tolerances, from the roundings that the header states (h = half a step of the
element type, u = 2^-24 for fp32):
  * scores: a dot product of D terms and the scale in fp32 are off by at most
    d = (D + 4) u scale sum |q k|; the exponential of an error d is a relative
    error of 2 d (d is small), and the exponential itself and the running sums
    add at most (n + 64) u;
  * every probability is rounded once to the element type: a relative h, in
    fp16 at least the half step 2^-25 of its smallest numbers (against a largest
    probability of 1 before the division);
  * the output is rounded once.
"""
import math

import pytest
import torch

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


class Case:
    """A batch with its pages anywhere in the pool and NaN wherever no
    position of a sequence lies."""

    def __init__(self, q_lens, kv_lens, Hq, Hk, D, page, dtype="bf16", seed=0, tree=None, spare=3, scale=None):
        g = torch.Generator().manual_seed(seed)
        dt = TYPES[dtype]
        self.q_lens, self.kv_lens, self.D, self.page = q_lens, kv_lens, D, page
        self.group = Hq // Hk
        need = [-(-max(0, n) // page) for n in kv_lens]
        total, width = sum(need) + spare, max(need + [1])
        order = torch.randperm(total, generator=g).to(torch.int32)
        self.table = torch.full((len(q_lens), width), -1, dtype=torch.int32)
        self.k = torch.full((total, page, Hk, D), math.nan, dtype=dt)
        self.v = torch.full((total, page, Hk, D), math.nan, dtype=dt)
        self.ks, self.vs, at = [], [], 0
        for b, n in enumerate(kv_lens):
            n = max(0, n)
            k, v = (torch.randn(n, Hk, D, generator=g).to(dt) for _ in range(2))
            self.ks.append(k)
            self.vs.append(v)
            for j in range(need[b]):
                p = int(order[at + j])
                self.table[b, j] = p
                m = min(page, n - j * page)
                self.k[p, :m], self.v[p, :m] = k[j * page:j * page + m], v[j * page:j * page + m]
            at += need[b]
        self.starts = [0]
        for n in q_lens:
            self.starts.append(self.starts[-1] + n)
        self.q = torch.randn(self.starts[-1], Hq, D, generator=g).to(dt)
        self.tree, self.scale = tree, D ** -0.5 if scale is None else scale
        self.Hq, self.Hk = Hq, Hk

    def inputs(self):
        t = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
        tree = None if self.tree is None else torch.tensor(
            [w - (1 << 64) if w >> 63 else w for w in self.tree], dtype=torch.int64, device=DEV)
        return dict(q=self.q.to(DEV), k_cache=self.k.to(DEV), v_cache=self.v.to(DEV), block_table=self.table.to(DEV),
                    q_starts=t(self.starts), kv_lens=t(self.kv_lens), max_q_len=max(self.q_lens + [0]),
                    scale=self.scale, tree_mask=tree)

    def check(self, out, lse, dtype):
        h = torch.finfo(dtype).eps / 2
        u = 2.0 ** -24
        assert out.dtype == dtype and not torch.isnan(out).any() and not torch.isnan(lse).any()
        for b, (m, n) in enumerate(zip(self.q_lens, self.kv_lens)):
            n = max(0, n)
            i, j = torch.arange(m, device=DEV)[:, None], torch.arange(n, device=DEV)[None, :]
            base = n - m
            if self.tree is None:
                sees = j <= base + i
            else:
                rows = self.tree[self.starts[b]:self.starts[b] + m]
                sees = torch.tensor([[c < base or (rows[r] >> (c - base)) & 1 for c in range(n)] for r in range(m)],
                                    dtype=torch.bool, device=DEV).view(m, n)
            for hq in range(self.Hq):
                q = self.q[self.starts[b]:self.starts[b] + m, hq].to(DEV).double()
                k = self.ks[b][:, hq // self.group].to(DEV).double()
                v = self.vs[b][:, hq // self.group].to(DEV).double()
                x = (q @ k.T * self.scale).masked_fill(~sees, -math.inf)
                top = x.amax(1, keepdim=True) if n else torch.full((m, 1), -math.inf, device=DEV, dtype=torch.double)
                top = torch.where(top == -math.inf, torch.zeros_like(top), top)
                p = torch.exp(x - top)
                total = p.sum(1, keepdim=True)
                want_lse = (total.log() + top)[:, 0]
                p = p / torch.where(total == 0, torch.ones_like(total), total)
                want = p @ v
                d = (self.D + 4) * u * self.scale * (q.abs() @ k.abs().T).amax(1, keepdim=True) if n else 0.0
                soft = 2 * d + (n + 64) * u
                size = p @ v.abs()
                tol = size * (h + soft) * 1.01 + h * want.abs()
                if dtype == torch.float16:  # its smallest steps: of the probabilities and of the output
                    tol = tol + 2.0 ** -25 * ((sees.double() @ v.abs()) / total.clamp_min(1) + 1)
                got = out[self.starts[b]:self.starts[b] + m, hq].double()
                off = (got - want).abs() - tol
                assert (off <= 0).all(), f"seq {b} head {hq}: {off.max().item():.3g} past the bound"
                got_lse = lse[self.starts[b]:self.starts[b] + m, hq].double()
                none = ~sees.any(1)
                assert (got_lse[none] == -math.inf).all() and (got[none] == 0).all()
                lse_tol = (soft + 8 * u * (1 + want_lse.abs())[:, None])[:, 0] if n else 0.0
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


def chain(*a, **k):
    return Case(*a, **k)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("D", [64, 128])
def test_types_pages_and_dims(dtype, page, D):
    run(Case([1, 5, 40], [77, 300, 40], 8, 2, D, page, dtype, seed=page + D))


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (2, 1), (5, 1), (8, 8), (20, 4), (14, 2), (48, 1), (64, 4)])
def test_head_layouts(Hq, Hk):
    run(Case([3, 1], [200, 129], Hq, Hk, 128, 64, seed=Hq))


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 383, 1023, 1025])
def test_lengths_of_one_token(n):
    run(Case([1], [n], 4, 1, 128, 16, seed=n))


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 2, 31, 32, 33, 64, 65, 100, 127, 128, 129, 256, 257, 400])
@pytest.mark.parametrize("before", [0, 1, 130])
def test_chunk_lengths(m, before):
    run(Case([m], [m + before], 4, 2, 64, 32, "fp16", seed=m))


@pytest.mark.gpu
def test_empty_sequences_and_rows_that_see_nothing():
    # no positions at all; a chunk longer than what the cache holds; a sequence without new tokens
    run(Case([1, 4, 0, 7, 3], [0, 2, 50, 7, 0], 4, 2, 128, 16))


@pytest.mark.gpu
def test_no_tokens():
    from weight_streaming_expert_gb300 import PagedAttention
    attn = PagedAttention(4, 2, 64, device=DEV)
    z = lambda *s, dt=torch.int32: torch.zeros(*s, dtype=dt, device=DEV)
    cache = z(2, 16, 2, 64, dt=torch.bfloat16)
    out = attn(z(0, 4, 64, dt=torch.bfloat16), cache, cache, z(0, 4), z(1), z(0), 0)
    assert out.shape == (0, 4, 64) and attn.status() == 0


@pytest.mark.gpu
def test_long_ragged_batch():
    run(Case([1] * 9, [5000, 1, 333, 4096, 17, 2048, 900, 3333, 64], 16, 2, 128, 16, seed=5))


@pytest.mark.gpu
def test_one_long_sequence():
    run(Case([6], [30001], 20, 4, 128, 64, seed=6))


@pytest.mark.gpu
def test_prompt_chunks():
    run(Case([700, 33, 1], [1500, 33, 900], 14, 2, 128, 32, "fp16", seed=7))
    run(Case([1030], [1030], 8, 1, 64, 64, "bf16", seed=8))


def random_tree(n, seed):
    g = torch.Generator().manual_seed(seed)
    seen = []
    for i in range(n):
        parent = int(torch.randint(-1, i, (1,), generator=g)) if i else -1
        seen.append((seen[parent] if parent >= 0 else 0) | (1 << i))
    return seen


@pytest.mark.gpu
@pytest.mark.parametrize("n,before", [(1, 10), (5, 0), (24, 100), (63, 129), (64, 1000), (64, 0)])
def test_trees(n, before):
    run(Case([n], [n + before], 8, 2, 64, 16, "fp16", seed=n, tree=random_tree(n, n)))
    run(Case([n, n], [n + before, n + 3], 6, 2, 128, 64, "bf16", seed=n,
             tree=random_tree(n, n) + random_tree(n, n + 1)))


@pytest.mark.gpu
def test_tree_rows_without_anything_to_see():
    tree = random_tree(12, 3)
    tree[0] = tree[7] = 0
    run(Case([12], [12], 4, 1, 128, 16, tree=tree))


@pytest.mark.gpu
def test_tree_of_a_chain_equals_the_chain():
    a = Case([40], [333], 8, 2, 128, 32, seed=9)
    b = Case([40], [333], 8, 2, 128, 32, seed=9, tree=[(2 << i) - 1 for i in range(40)])
    assert torch.equal(run(a), run(b))


@pytest.mark.gpu
def test_large_scores():
    # one position takes it all, and the running maximum climbs along the way
    c = Case([3, 1], [700, 515], 4, 2, 128, 64, seed=10, scale=1.5)
    for b in range(2):
        ramp = torch.linspace(0.1, 6, c.kv_lens[b])[:, None, None]
        c.ks[b].copy_((c.ks[b].float() * ramp).to(torch.bfloat16))
        for j in range(-(-c.kv_lens[b] // 64)):
            p, m = int(c.table[b, j]), min(64, c.kv_lens[b] - 64 * j)
            c.k[p, :m] = c.ks[b][64 * j:64 * j + m]
    run(c)


@pytest.mark.gpu
def test_infinite_keys_of_hidden_positions():
    """A hidden position's key may hold anything: infinities and NaN."""
    c = Case([8], [100], 4, 2, 64, 16, "fp16", seed=11, tree=[1 << i for i in range(8)])
    x = c.inputs()
    for i, bad in ((3, math.nan), (5, math.inf), (7, -math.inf)):
        pos = 92 + i
        x["k_cache"][int(c.table[0, pos // 16]), pos % 16] = bad
    from weight_streaming_expert_gb300 import PagedAttention
    attn = PagedAttention(4, 2, 64, device=DEV)
    out, lse = attn(return_lse=True, **x)
    clean, clean_lse = attn(return_lse=True, **c.inputs())
    keep = [0, 1, 2, 4, 6]  # the rows that do not see those positions
    assert torch.equal(out[keep], clean[keep]) and torch.equal(lse[keep], clean_lse[keep])


@pytest.mark.gpu
def test_strides_orders_and_given_outputs():
    c = Case([3, 20], [100, 257], 6, 2, 128, 32, seed=12)
    plain = run(c)
    x = c.inputs()
    T = c.q.shape[0]
    wide = torch.full((T, 10, 2 * 128), math.nan, dtype=torch.bfloat16, device=DEV)
    wide[:, 2:8, 128:] = x["q"]
    pools = torch.full((2, x["k_cache"].shape[0], 2, 32, 2, 128), math.nan, dtype=torch.bfloat16, device=DEV)
    pools[0, :, 1], pools[1, :, 0] = x["k_cache"], x["v_cache"]
    rows = torch.full((2, x["block_table"].shape[1] + 3), 1 << 30, dtype=torch.int32, device=DEV)
    rows[:, :-3] = x["block_table"]
    out = torch.full((T, 9, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    x.update(q=wide[:, 2:8, 128:], k_cache=pools[0, :, 1], v_cache=pools[1, :, 0], block_table=rows, out=out[:, 1:7])
    got = run(c, **{k: x[k] for k in ("q", "k_cache", "v_cache", "block_table", "out")})
    assert torch.equal(got, plain)
    assert (out[:, 0] == 7).all() and (out[:, 7:] == 7).all()
    # heads outermost in memory
    turned = c.q.to(DEV).transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(run(c, q=turned), plain)


@pytest.mark.gpu
def test_cache_beyond_32_bit_offsets():
    """Pages past 2^31 elements (and past 2^32 bytes) of the pool."""
    page, Hk, D = 256, 8, 128
    n_pages = (1 << 32) // (page * Hk * D) // 2 * 2 + 40  # > 2^32 elements
    k = torch.empty((n_pages, page, Hk, D), dtype=torch.bfloat16, device=DEV)
    v = torch.empty_like(k)
    c = Case([2], [600], 16, Hk, D, page, seed=13)
    for j in range(3):
        far = n_pages - 1 - 2 * j
        old = int(c.table[0, j])
        k[far], v[far] = c.k[old].to(DEV), c.v[old].to(DEV)
        c.table[0, j] = far
    run(c, k_cache=k, v_cache=v)


@pytest.mark.gpu
def test_graph_replay_other_stream_and_changed_lengths():
    """A captured call reads lengths and tables when it is replayed."""
    from weight_streaming_expert_gb300 import PagedAttention
    a = Case([6, 6], [500, 333], 20, 4, 128, 64, seed=14)
    b = Case([6, 6], [80, 450], 20, 4, 128, 64, seed=15, spare=3)
    attn = PagedAttention(20, 4, 128, device=DEV)
    pages = max(a.k.shape[0], b.k.shape[0])
    x = a.inputs()

    def padded(c):
        y = c.inputs()
        for n in ("k_cache", "v_cache"):
            t = torch.full((pages,) + tuple(y[n].shape[1:]), math.nan, dtype=y[n].dtype, device=DEV)
            t[:y[n].shape[0]] = y[n]
            y[n] = t
        t = torch.full((2, 8), -1, dtype=torch.int32, device=DEV)
        t[:, :y["block_table"].shape[1]] = y["block_table"]
        y["block_table"] = t
        return y

    x = padded(a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    attn(return_lse=True, stream=s, **x)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out, lse = attn(return_lse=True, stream=s, **x)
    for case in (a, b, a):
        for n, t in padded(case).items():
            if torch.is_tensor(t):
                x[n].copy_(t)
        g.replay()
        torch.cuda.synchronize()
        case.check(out, lse, torch.bfloat16)
    assert attn.status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hk", [(3, 3), (12, 6), (16, 16), (128, 1), (96, 2), (100, 1)])
def test_more_head_layouts(Hq, Hk):
    # heads that neighbouring CTAs share out, and groups of which one token fills a tile
    run(Case([2, 5, 1], [300, 70, 513], Hq, Hk, 64, 16, "fp16", seed=Hq))


@pytest.mark.gpu
@pytest.mark.parametrize("batch,q_len", [(33, 1), (100, 3), (300, 1), (40, 30)])
def test_many_sequences(batch, q_len):
    g = torch.Generator().manual_seed(batch)
    lens = torch.randint(0, 400, (batch,), generator=g).tolist()
    q = torch.randint(0, q_len + 1, (batch,), generator=g).tolist()
    run(Case(q, [max(n, m) if i % 7 else n for i, (n, m) in enumerate(zip(lens, q))], 8, 2, 64, 32, seed=batch))


@pytest.mark.gpu
@pytest.mark.parametrize("batch", [1, 2, 7, 23, 61, 90])
def test_shares_that_end_anywhere_in_an_item(batch):
    """Items of one to some units, so that the CTAs' shares end before, at and
    behind the first unit of one."""
    g = torch.Generator().manual_seed(batch)
    draw = lambda lo, hi: int(torch.randint(lo, hi, (1,), generator=g))
    q_lens = [draw(20, 260) for _ in range(batch)]
    q_lens[0] = 259
    run(chain(q_lens, [m + draw(-10, 600) for m in q_lens], 4, 2, 64, 32, "fp16", batch))


@pytest.mark.gpu
def test_one_handle_over_calls_of_every_kind():
    """What a call leaves in the handle's workspace is not another's."""
    from weight_streaming_expert_gb300 import PagedAttention
    attn = PagedAttention(8, 2, 128, device=DEV)
    cases = [Case([6, 6], [4000, 900], 8, 2, 128, 64, seed=1), Case([0, 6], [4000, 20], 8, 2, 128, 64, seed=2),
             Case([300], [2000], 8, 2, 128, 16, "fp16", seed=3), Case([1] * 90, [700] * 90, 8, 2, 128, 32, seed=4),
             Case([64, 0, 2], [64, 500, 5000], 8, 2, 128, 16, seed=5), Case([6, 6], [4000, 0], 8, 2, 128, 64, seed=6)]
    for c in cases + cases[::-1]:
        out, lse = attn(return_lse=True, **c.inputs())
        assert attn.status() == 0
        c.check(out, lse, c.q.dtype)


@pytest.mark.gpu
def test_same_bits_every_time():
    c = Case([1] * 7, [3000, 2, 800, 1500, 77, 4000, 129], 32, 4, 128, 16, seed=16)
    first = run(c)
    for _ in range(3):
        assert torch.equal(run(c), first)


@pytest.mark.gpu
def test_bad_pages_and_lengths_are_reported():
    from weight_streaming_expert_gb300 import PagedAttention
    from weight_streaming_expert_gb300 import native as N
    c = Case([2, 2], [100, 90], 4, 2, 128, 32, seed=17)
    attn = PagedAttention(4, 2, 128, device=DEV)
    x = c.inputs()
    for bad in (-1, c.k.shape[0], 1 << 30):
        table = x["block_table"].clone()
        table[0, 1] = bad
        out = attn(**{**x, "block_table": table})
        assert attn.status() == N.MOE_ERR_INVALID_ARG and "page" in N.last_error()
        assert torch.isfinite(out).all() and attn.status() == 0
    good = attn(**x)
    lens = torch.tensor([100, 10000], dtype=torch.int32, device=DEV)
    table = x["block_table"].clamp_min(0)
    out = attn(**{**x, "kv_lens": lens, "block_table": table})
    assert attn.status() == N.MOE_ERR_INVALID_ARG and "length" in N.last_error()
    assert torch.equal(out[:2], good[:2])


def args(**change):
    from weight_streaming_expert_gb300 import native as N
    a = N.moe_attn_args_t()
    base = dict(dtype=0, batch=1, n_tokens=1, max_q_len=1, scale=1.0, q=16, q_token_stride=256, q_head_stride=64,
                k_cache=16, v_cache=16, k_page_stride=1024, k_row_stride=64, v_page_stride=1024, v_row_stride=64,
                n_pages=4, page_size=16, block_table=16, table_stride=4, q_starts=16, kv_lens=16, tree_mask=None,
                out=16, out_token_stride=256, out_head_stride=64, lse=None)
    for k, v in {**base, **change}.items():
        setattr(a, k, v)
    return a


REFUSED = [("dtype", 2, 1, "dtype"), ("batch", -1, 1, "batch"), ("n_tokens", -1, 1, "n_tokens"),
           ("scale", 0.0, 1, "scale"), ("scale", -1.0, 1, "scale"), ("scale", math.inf, 1, "scale"),
           ("scale", math.nan, 1, "scale"), ("page_size", 0, 2, "page_size"), ("page_size", 48, 2, "page_size"),
           ("page_size", 8, 2, "page_size"), ("n_pages", 0, 1, "n_pages"), ("q", None, 1, "null"),
           ("q", 8, 1, "aligned"),
           ("k_cache", 24, 1, "aligned"), ("v_cache", None, 1, "null"), ("out", 20, 1, "aligned"),
           ("block_table", None, 1, "block_table"), ("q_starts", 2, 1, "q_starts"), ("kv_lens", None, 1, "kv_lens"),
           ("q_token_stride", 4, 1, "stride"), ("k_row_stride", 65, 1, "stride"), ("v_page_stride", 1, 1, "stride"),
           ("lse", 2, 1, "aligned")]


@pytest.mark.parametrize("field,value,status,word", REFUSED)
def test_refusals(field, value, status, word):
    import ctypes

    from weight_streaming_expert_gb300 import native as N
    L = N.lib()
    fake = ctypes.create_string_buffer(4096)  # refused before the handle is looked at
    rc = L.moe_attn_forward(ctypes.cast(fake, ctypes.c_void_p), ctypes.byref(args(**{field: value})), None)
    assert rc == status and word in N.last_error()


def test_more_refusals():
    import ctypes

    from weight_streaming_expert_gb300 import native as N
    L = N.lib()
    assert L.moe_attn_forward(None, ctypes.byref(args()), None) == N.MOE_ERR_INVALID_ARG
    fake = ctypes.cast(ctypes.create_string_buffer(4096), ctypes.c_void_p)
    assert L.moe_attn_forward(fake, None, None) == N.MOE_ERR_INVALID_ARG
    assert L.moe_attn_forward(fake, ctypes.byref(args(tree_mask=16, max_q_len=65)), None) == N.MOE_ERR_UNSUPPORTED
    assert L.moe_attn_forward(fake, ctypes.byref(args(n_tokens=0, q=None)), None) == N.MOE_OK
    for bad in ((0, 1, 64), (3, 2, 64), (4, 0, 64), (4, 2, 96), (4, 2, 0)):
        assert not L.moe_attn_create(*bad) and N.last_error()
    assert L.moe_attn_get_status(None) == N.MOE_ERR_INVALID_ARG
    L.moe_attn_destroy(None)


@pytest.mark.gpu
def test_python_refusals():
    from weight_streaming_expert_gb300 import PagedAttention
    c = Case([2], [40], 4, 2, 64, 16)
    attn = PagedAttention(4, 2, 64, device=DEV)
    x = c.inputs()
    bad = dict(q=[x["q"].float(), x["q"][:, :3], x["q"].transpose(1, 2), x["q"].cpu()],
               k_cache=[x["k_cache"].half(), x["k_cache"][:, :, :1], x["k_cache"][..., :32]],
               block_table=[x["block_table"].long(), x["block_table"][0]],
               q_starts=[x["q_starts"].long(), x["kv_lens"]],
               kv_lens=[x["q_starts"]], tree_mask=[torch.zeros(3, dtype=torch.int64, device=DEV)],
               out=[torch.empty(2, 4, 64, device=DEV), torch.empty(1, 4, 64, dtype=torch.bfloat16, device=DEV)])
    for name, values in bad.items():
        for v in values:
            with pytest.raises(ValueError):
                attn(**{**x, name: v})


@pytest.mark.gpu
def test_a_closed_handle_is_refused():
    from weight_streaming_expert_gb300 import PagedAttention
    from weight_streaming_expert_gb300.native import MoEError
    c = Case([2], [40], 4, 2, 64, 16)
    attn = PagedAttention(4, 2, 64, device=DEV)
    attn(**c.inputs())
    torch.cuda.synchronize()
    attn.close()
    attn.close()
    with pytest.raises(MoEError):
        attn(**c.inputs())
    assert attn.status() != 0
