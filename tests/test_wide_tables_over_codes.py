"""Chunks over codes whose block table is much wider than its sequences (the
fixed table of a captured graph): their pages are unpacked by the lengths, in
turns where the table's width times the batch exceeds what is kept at a time.
Tolerances: those of test_quantised_attention and test_shared_prefix."""
import pytest
import torch

from tests.test_quantised_attention import DEV, CodeCase
from tests.test_shared_prefix import Shared


def widened(table, width):
    wide = torch.full((table.shape[0], width), -1, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = table
    return wide


@pytest.mark.gpu
@pytest.mark.parametrize("width", [100, 5000, 40000])
@pytest.mark.parametrize("prefix", [0, 96])
def test_wide_tables(width, prefix):
    from weight_streaming_expert_gb300 import PagedAttention
    q_lens, own = [40, 1, 0, 90, 17], [700, 1, 33, 90, 230]
    if prefix:
        case = Shared(q_lens, own, prefix, 8, 4, 128, 16, seed=width, codes=True)
    else:
        case = CodeCase(q_lens, own, 8, 4, 128, 16, seed=width)
    x = case.inputs()
    x["block_table"] = widened(x["block_table"], width)
    attn = PagedAttention(8, 4, 128, device=DEV)
    out, lse = attn(return_lse=True, **x)
    assert attn.status() == 0
    case.check(out, lse, torch.bfloat16)
    assert torch.equal(attn(**x), out)
    # a view as narrow as the longest sequence takes less room for the same
    x["block_table"] = x["block_table"][:, :-(-(prefix + 700) // 16)]
    out, lse = attn(return_lse=True, **x)
    assert attn.status() == 0
    case.check(out, lse, torch.bfloat16)
    attn.close()


@pytest.mark.gpu
def test_captured_with_a_wide_table_and_lengths_that_grow():
    from weight_streaming_expert_gb300 import PagedAttention
    case = CodeCase([70, 20], [2500, 900], 4, 1, 64, 32, "fp16", seed=8)
    x = case.inputs()
    x["block_table"] = widened(x["block_table"], 3000)
    attn = PagedAttention(4, 1, 64, device=DEV)
    lens = x["kv_lens"].clone()
    out = torch.empty_like(x["q"])
    x["kv_lens"].fill_(100)
    attn(out=out, **x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attn(out=out, **x)
    x["kv_lens"].copy_(lens)
    graph.replay()
    want, lse = attn(return_lse=True, **x)
    assert attn.status() == 0 and torch.equal(out, want)
    case.check(want, lse, torch.float16)
    attn.close()
