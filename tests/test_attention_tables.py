"""Block tables and lengths of other shapes than a full, contiguous table with
ascending starts: a table that sequences share, a view of a wider one, starts
that make no sense."""
import math

import pytest
import torch

from tests.test_attention import DEV, Case, args

INT_MIN = -2 ** 31


def outputs(c, attn=None, **change):
    from weight_streaming_expert_gb300 import PagedAttention
    attn = attn or PagedAttention(c.Hq, c.Hk, c.D, device=DEV)
    return attn(return_lse=True, **{**c.inputs(), **change})


@pytest.mark.gpu
@pytest.mark.parametrize("q_lens,n", [([1, 1, 1], 300), ([4, 2], 700), ([90, 40], 95)])
def test_a_table_that_all_sequences_share(q_lens, n):
    from weight_streaming_expert_gb300 import PagedAttention
    c = Case(q_lens, [n] * len(q_lens), 8, 2, 128, 16, seed=n)
    attn = PagedAttention(8, 2, 128, device=DEV)
    one = c.inputs()["block_table"][:1]
    copied = one.repeat(len(q_lens), 1)
    out, lse = outputs(c, attn, block_table=copied)
    assert attn.status() == 0 and lse.isfinite().all()
    got, got_lse = outputs(c, attn, block_table=one.expand(len(q_lens), -1))
    assert attn.status() == 0
    assert torch.equal(got, out) and torch.equal(got_lse, lse)


@pytest.mark.gpu
def test_a_length_past_the_width_of_a_view():
    """It is cut and reported; what lies beside the view is not read."""
    from weight_streaming_expert_gb300 import PagedAttention
    from weight_streaming_expert_gb300 import native as N
    c = Case([2, 3], [64, 64], 4, 2, 64, 16, "fp16", seed=1)
    attn = PagedAttention(4, 2, 64, device=DEV)
    x = c.inputs()
    wide = torch.full((2, 11), 1 << 30, dtype=torch.int32, device=DEV)  # no pages of this cache
    wide[:, 3:7] = x["block_table"]
    out, lse = outputs(c, attn, block_table=wide[:, 3:7])
    assert attn.status() == 0 and torch.equal(out, outputs(c, attn)[0])
    for lens in ([64, 65], [80, 64], [64, 1 << 30]):
        kv_lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        got, _ = outputs(c, attn, block_table=wide[:, 3:7], kv_lens=kv_lens)
        assert attn.status() == N.MOE_ERR_INVALID_ARG
        assert "length" in N.last_error() and "page" not in N.last_error()
        assert got.isfinite().all()


@pytest.mark.gpu
def test_a_table_without_columns():
    from weight_streaming_expert_gb300 import PagedAttention
    from weight_streaming_expert_gb300 import native as N
    c = Case([2, 1], [0, 0], 4, 2, 64, 16, seed=2)
    attn = PagedAttention(4, 2, 64, device=DEV)
    for B in (1, 2):
        i = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
        empty = torch.zeros(B, 0, dtype=torch.int32, device=DEV)
        starts = i(0, 3) if B == 1 else i(0, 2, 3)
        out, lse = outputs(c, attn, block_table=empty, q_starts=starts, kv_lens=i(*[0] * B), max_q_len=3)
        assert attn.status() == 0 and (out == 0).all() and (lse == -math.inf).all()
        outputs(c, attn, block_table=empty, q_starts=starts, kv_lens=i(*[9] * B), max_q_len=3)
        assert attn.status() == N.MOE_ERR_INVALID_ARG


def test_refusals_of_tables():
    import ctypes

    from weight_streaming_expert_gb300 import native as N
    fake = ctypes.cast(ctypes.create_string_buffer(4096), ctypes.c_void_p)
    call = lambda **k: N.lib().moe_attn_forward(fake, ctypes.byref(args(**k)), None)
    assert call(table_pages=-1) == N.MOE_ERR_INVALID_ARG and "table_pages" in N.last_error()
    assert call(table_stride=-1) == N.MOE_ERR_INVALID_ARG and "table_stride" in N.last_error()
    assert call(table_pages=1, block_table=None) == N.MOE_ERR_INVALID_ARG and "block_table" in N.last_error()


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["chain", "tree", "chunk"])
def test_starts_that_make_no_sense(form):
    """They are reported; rows past the last token are not touched, and the
    sequences whose starts are right keep their results."""
    from weight_streaming_expert_gb300 import PagedAttention
    from weight_streaming_expert_gb300 import native as N
    lens = [90, 40] if form == "chunk" else [3, 2]
    tree = [1, 3, 5, 1, 3] if form == "tree" else None
    c = Case(lens, [200, 150], 8, 2, 64, 16, "fp16", seed=3, tree=tree)
    T, first = sum(lens), lens[0]
    attn = PagedAttention(8, 2, 64, device=DEV)
    good, _ = outputs(c, attn)
    assert attn.status() == 0
    for starts, right in (([0, first, INT_MIN], True), ([0, first, INT_MIN + first - 1], True),
                          ([0, first, -1], True), ([0, first, 1], True), ([INT_MIN, first, T], False),
                          ([0, 2 ** 31 - 1, T], False), ([2 ** 31 - 1, INT_MIN, 2 ** 31 - 1], False),
                          ([-5, T + 7, INT_MIN], False), ([T, T, T + 1], False)):
        out = torch.full((2 * T + 300, 8, 64), 7.0, dtype=torch.float16, device=DEV)
        outputs(c, attn, q_starts=torch.tensor(starts, dtype=torch.int32, device=DEV), out=out[:T])
        assert attn.status() == N.MOE_ERR_INVALID_ARG and "length" in N.last_error(), starts
        assert (out[T:] == 7).all() and out.isfinite().all(), starts
        if right:
            assert torch.equal(out[:first], good[:first]), starts


@pytest.mark.gpu
def test_many_heads_over_one_in_a_long_table():
    """A table of a million positions does not make a chunk too much work: 128
    heads of a token fill a tile, so 8192 tokens are 4096 items of at most 8192
    tiles of positions."""
    from weight_streaming_expert_gb300 import PagedAttention
    g = torch.Generator(device=DEV).manual_seed(4)
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV).bfloat16()
    T, page = 8192, 64
    q, k, v = rand(T, 128, 64), rand(T // page, page, 1, 64), rand(T // page, page, 1, 64)
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    narrow = torch.arange(T // page, dtype=torch.int32, device=DEV)[None]
    wide = torch.full((1, (1 << 20) // page), -1, dtype=torch.int32, device=DEV)
    wide[:, :T // page] = narrow
    attn = PagedAttention(128, 1, 64, device=DEV)
    want = attn(q, k, v, narrow, i(0, T), i(T), T)
    got = attn(q, k, v, wide, i(0, T), i(T), T)
    assert attn.status() == 0 and torch.equal(got, want)


@pytest.mark.gpu
def test_too_much_work_is_refused():
    from weight_streaming_expert_gb300 import PagedAttention
    from weight_streaming_expert_gb300 import native as N
    attn = PagedAttention(64, 64, 64, device=DEV)
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device=DEV)
    table = z(1, 1, dt=torch.int32).expand(1, 1 << 22)  # 2^30 positions: 2^23 tiles
    q = z(1024, 64, 64)  # 4 items of 64 heads
    with pytest.raises(N.MoEError, match="too much work"):
        attn(q, z(1, 256, 64, 64), z(1, 256, 64, 64), table.contiguous(), z(2, dt=torch.int32), z(1, dt=torch.int32),
             1024)


@pytest.mark.gpu
@pytest.mark.parametrize("batch,T,Hq,Hk,positions", [(4096, 4096, 8, 2, 1 << 24), (32, 256, 20, 5, 1 << 30)])
def test_overlapping_chunks_that_are_too_much_work(batch, T, Hq, Hk, positions):
    """Every second sequence names all tokens, over all positions that its row
    of the table could hold: more work than 32 bits count, of which nothing is
    done."""
    from weight_streaming_expert_gb300 import PagedAttention
    from weight_streaming_expert_gb300 import native as N
    attn = PagedAttention(Hq, Hk, 64, device=DEV)
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=DEV)
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    k = z(2, 256, Hk, 64)
    table = torch.zeros(1, positions // 256, dtype=torch.int32, device=DEV).expand(batch, -1)
    starts = torch.zeros(batch + 1, dtype=torch.int32, device=DEV)
    starts[1::2] = T
    lens = torch.full((batch,), positions, dtype=torch.int32, device=DEV)
    out = torch.full((T, Hq, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    attn(z(T, Hq, 64), k, k, table, starts, lens, T, out=out)
    assert attn.status() == N.MOE_ERR_INVALID_ARG and "length" in N.last_error()
    assert (out == 7).all()
    # without the overlap the same tables are fine
    starts[1:] = T
    lens.fill_(300)
    lens[0] = T
    attn(z(T, Hq, 64), k, k, table, starts, lens, T, out=out)
    assert attn.status() == 0 and (out == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("batch", [2, 200])
def test_a_longest_chunk_of_zero_is_reported(batch):
    """As any other number that is smaller than a chunk."""
    from weight_streaming_expert_gb300 import PagedAttention
    from weight_streaming_expert_gb300 import native as N
    c = Case([2] * batch, [30] * batch, 4, 2, 64, 16, seed=5)
    attn = PagedAttention(4, 2, 64, device=DEV)
    for longest in (1, 0):
        outputs(c, attn, max_q_len=longest)
        assert attn.status() == N.MOE_ERR_INVALID_ARG and "max_q_len" in N.last_error()
    empty = torch.zeros(batch + 1, dtype=torch.int32, device=DEV)  # no chunk has a token
    outputs(c, attn, max_q_len=0, q_starts=empty)
    assert attn.status() == 0
