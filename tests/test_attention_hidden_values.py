"""A row's output is the sum over the positions that it sees: the values of
others -- later tokens of its chunk, other branches of a tree -- may hold
anything, infinities and NaN among them.

A case is computed twice, with finite values everywhere and with some values
replaced.  Columns of a row in which it sees a replaced value follow the formula
(NaN, or the infinity, or NaN of both); all others repeat the first call's
bits."""
import math

import pytest
import torch

from tests.test_attention import DEV, Case, random_tree

pytestmark = pytest.mark.gpu


def check(c, bad, attn=None):
    """bad: (sequence, position, columns, value) of every value head."""
    from weight_streaming_expert_gb300 import PagedAttention
    attn = attn or PagedAttention(c.Hq, c.Hk, c.D, device=DEV)
    clean, clean_lse = attn(return_lse=True, **c.inputs())
    x = c.inputs()
    for b, pos, columns, value in bad:
        x["v_cache"][int(c.table[b, pos // c.page]), pos % c.page, :, columns] = value
    out, lse = attn(return_lse=True, **x)
    assert attn.status() == 0
    assert torch.equal(lse, clean_lse)
    want = clean.double()
    for b, pos, columns, value in bad:
        m, base = c.q_lens[b], c.kv_lens[b] - c.q_lens[b]
        for i in range(m):
            row = c.starts[b] + i
            sees = pos <= base + i if c.tree is None else pos < base or (c.tree[row] >> (pos - base)) & 1
            if sees:
                want[row, :, columns] += value
    want = want.to(out.dtype)
    same = (out == want) | (out.isnan() & want.isnan())
    assert same.all(), f"{int((~same).sum())} elements differ, first {(~same).nonzero()[0].tolist()}"


ALL = slice(None)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64)])
@pytest.mark.parametrize("before", [0, 70, 3000])
def test_a_chain(dtype, D, before):
    c = Case([6], [6 + before], 20, 4, D, 16, dtype, seed=before)
    for i in range(6):
        check(c, [(0, before + i, ALL, math.nan)])
    check(c, [(0, before + 2, slice(3, 9), math.inf), (0, before + 4, slice(5, 40), -math.inf)])


@pytest.mark.parametrize("Hq,Hk,D", [(8, 2, 64), (8, 2, 128), (4, 4, 128), (20, 1, 64)])
@pytest.mark.parametrize("n,before", [(24, 0), (24, 100), (64, 1000), (64, 3)])
def test_branches_of_a_tree(Hq, Hk, D, n, before):
    tree = random_tree(n, n) + random_tree(n, n + 1)
    c = Case([n, n], [n + before, n + before + 9], Hq, Hk, D, 16, "fp16" if D == 64 else "bf16", seed=n, tree=tree)
    check(c, [(0, before + i, ALL, math.nan) for i in (1, n - 1)])
    check(c, [(1, before + 9 + i, slice(i, i + 7), (math.inf, -math.inf, math.nan)[i % 3]) for i in range(n)])


@pytest.mark.parametrize("before", [0, 40, 130])
def test_rows_of_a_tree_that_see_nothing(before):
    tree = [1 << i for i in range(12)]
    if before == 0:
        tree[0] = tree[7] = 0
    c = Case([12], [12 + before], 4, 1, 128, 16, tree=tree)
    check(c, [(0, before + i, ALL, math.nan) for i in range(12) if i not in (3, 8)])


@pytest.mark.parametrize("Hq,Hk", [(8, 1), (2, 2), (5, 1), (100, 1)])
@pytest.mark.parametrize("D,dtype", [(64, "fp16"), (128, "bf16")])
@pytest.mark.parametrize("m,before", [(257, 0), (700, 33), (300, 2000)])
def test_later_tokens_of_a_chunk(Hq, Hk, D, dtype, m, before):
    c = Case([m], [m + before], Hq, Hk, D, 64, dtype, seed=m + Hq)
    last = m + before - 1
    check(c, [(0, last, ALL, math.nan)])
    check(c, [(0, before + m // 2, ALL, math.nan), (0, before + m // 3, slice(0, 8), math.inf)])
    check(c, [(0, before + i, slice(i % D, i % D + 1), math.inf) for i in range(1, m, 37)])


def test_a_chunk_longer_than_the_cache():
    """Its first tokens see nothing."""
    c = Case([40, 300], [25, 140], 4, 1, 64, 16, "fp16", seed=5)
    check(c, [(0, 3, ALL, math.nan), (1, 77, slice(1, 30), -math.inf)])


def test_batches_and_one_handle():
    """A call with such values leaves nothing behind for the next."""
    from weight_streaming_expert_gb300 import PagedAttention
    attn = PagedAttention(8, 2, 128, device=DEV)
    a = Case([200, 1, 33, 6], [900, 300, 33, 1000], 8, 2, 128, 32, seed=1)
    b = Case([5] * 40, [400 + i for i in range(40)], 8, 2, 128, 32, seed=2)
    for _ in range(2):
        check(a, [(0, 850, ALL, math.nan), (2, 20, ALL, math.inf), (3, 997, slice(0, 1), math.nan)], attn)
        check(b, [(i, 398 + i, ALL, math.nan) for i in range(0, 40, 3)], attn)


@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "fp16")])
def test_many_short_items_in_a_row(D, dtype):
    """A CTA goes through many items of one tile of positions."""
    g = torch.Generator().manual_seed(7)
    q_lens = torch.randint(33, 64, (600,), generator=g).tolist()
    c = Case(q_lens, [m + m % 60 for m in q_lens], 16, 4, D, 16, dtype, seed=3)
    check(c, [(b, c.kv_lens[b] - 1 - b % 30, ALL if b % 3 else slice(0, 9), math.nan) for b in range(0, 600, 2)])
    check(c, [(b, c.kv_lens[b] - 2, ALL, math.inf) for b in range(600)])
