"""Pages that a block table names outside a quantised cache: their positions
count as zeros, whatever lay in the kernel's tiles before them.  Tolerances:
those of test_quantised_attention, a missing row being one of zeros whose scale
is the least there is."""
import pytest
import torch

from tests.test_quantised_attention import DEV, CodeCase


def missing(B, n, m, D, Hq):
    """Every second sequence has values around 2^30, the others a page or two
    that are not there."""
    case = CodeCase([m] * B, [n] * B, Hq, 1, D, 16, seed=B + n)
    gone = []
    for b in range(B):
        pages = case.table[b, :-(-n // 16)].long()
        if b % 2 == 0:
            case.scales["v"][pages] += 30
        else:
            gone.append((b, [b % 3, 5 + b % 7]))
    case.read_codes()
    for b, places in gone:
        for j in places:
            case.table[b, j] = (1 << 20) + b if b % 4 == 1 else -1 - b
            rows = slice(j * 16, j * 16 + 16)
            case.ks[b][rows], case.vs[b][rows], case.fs[b][rows] = 0, 0, -40
    return case


@pytest.mark.gpu
@pytest.mark.parametrize("D,m,Hq", [(128, 1, 4), (64, 1, 1), (64, 2, 8), (128, 4, 8), (64, 5, 12), (64, 20, 4)])
def test_a_missing_page_counts_as_zeros(D, m, Hq):
    from weight_streaming_expert_gb300 import PagedAttention
    from weight_streaming_expert_gb300 import native as N
    case = missing(300, 700, m, D, Hq)
    attn = PagedAttention(Hq, 1, D, device=DEV)
    x = case.inputs()
    out, lse = attn(return_lse=True, **x)
    assert attn.status() == N.MOE_ERR_INVALID_ARG and "page" in N.last_error()
    case.check(out, lse, torch.bfloat16)
    assert torch.equal(attn(**x), out)
    attn.close()
