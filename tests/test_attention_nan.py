"""A NaN in a query or in keys that are seen has to show in the outputs,
however the work is shared out.

One sequence and one key/value head: every 128 positions are a CTA's share, so
100 positions stay in one piece, 300 are joined from three parts and 1200 from
ten; 3 tokens of 4 heads take the form for few rows, 40 the one for many."""
import math

import pytest
import torch

from tests.test_attention import DEV, Case

pytestmark = pytest.mark.gpu
FORMS = [(m, n) for m in (3, 40) for n in (100, 300, 1200)]


def outputs(c, **change):
    from weight_streaming_expert_gb300 import PagedAttention
    attn = PagedAttention(c.Hq, c.Hk, c.D, device=DEV)
    got = attn(return_lse=True, **{**c.inputs(), **change})
    assert attn.status() == 0
    return got


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64)])
@pytest.mark.parametrize("m,n", FORMS)
def test_a_query_that_is_not_a_number(m, n, dtype, D):
    c = Case([m], [n], 4, 1, D, 16, dtype, seed=n + m)
    out, lse = outputs(c)
    q = c.q.to(DEV)
    q[1, 2, 5] = math.nan
    got, got_lse = outputs(c, q=q)
    assert got[1, 2].isnan().all() and got_lse[1, 2].isnan()
    rest = torch.ones(m, 4, dtype=torch.bool, device=DEV)
    rest[1, 2] = False
    assert torch.equal(got[rest], out[rest]) and torch.equal(got_lse[rest], lse[rest])


@pytest.mark.parametrize("m,n", FORMS)
def test_keys_that_are_not_numbers_over_a_whole_share(m, n):
    c = Case([m], [n], 4, 1, 128, 16, seed=n + m)
    for first in range(0, n, 128):
        k = c.k.to(DEV)
        at = torch.arange(first, min(n, first + 128))
        k[c.table[0, at // 16].long().to(DEV), (at % 16).to(DEV)] = math.nan
        out, lse = outputs(c, k_cache=k)
        sees = torch.arange(m) + n - m >= first  # those that see any of them
        assert out[sees.to(DEV)].isnan().all() and lse[sees.to(DEV)].isnan().all()
        assert out[~sees.to(DEV)].isfinite().all() and lse[~sees.to(DEV)].isfinite().all()


@pytest.mark.parametrize("m,n", FORMS)
def test_one_key_that_is_not_a_number(m, n):
    c = Case([m], [n], 4, 1, 64, 32, "fp16", seed=n + m)
    out, lse = outputs(c)
    for pos in (0, n // 2, n - 1):
        k = c.k.to(DEV)
        k[int(c.table[0, pos // 32]), pos % 32, 0, 7] = math.nan
        got, got_lse = outputs(c, k_cache=k)
        sees = (torch.arange(m) + n - m >= pos).to(DEV)
        assert got[sees].isnan().all() and got_lse[sees].isnan().all()
        assert torch.equal(got[~sees], out[~sees]) and torch.equal(got_lse[~sees], lse[~sees])


@pytest.mark.parametrize("m,n", FORMS)
def test_a_seen_value_that_is_not_finite(m, n):
    """Its column and no other, of the rows that see it."""
    c = Case([m], [n], 4, 1, 128, 16, seed=n + m)
    out, lse = outputs(c)
    for pos, bad in ((0, math.nan), (n - m, math.inf), (n // 2, -math.inf)):
        v = c.v.to(DEV)
        v[int(c.table[0, pos // 16]), pos % 16, 0, 33] = bad
        got, got_lse = outputs(c, v_cache=v)
        sees = (torch.arange(m) + n - m >= pos).to(DEV)
        assert sees.all()
        column = got[:, :, 33]
        assert column.isnan().all() if bad != bad else (column == bad).all()
        other = [i for i in range(128) if i != 33]
        assert torch.equal(got[:, :, other], out[:, :, other]) and torch.equal(got_lse, lse)
