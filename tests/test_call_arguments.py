"""What is no tensor, or a tensor of another number of dimensions, is named in a
ValueError by every call."""
import pytest
import torch

from tests.test_attention import DEV, Case

NO_TENSORS = (None, [1.0, 2.0], 3)


def bad_calls(call, good, names, optional=()):
    """Each argument in turn replaced by what does not fit."""
    for name in names:
        for value in NO_TENSORS:
            if value is None and name in optional:
                continue
            with pytest.raises(ValueError, match=name):
                call(**{**good, name: value})


def test_logits_that_are_no_tensor():
    from weight_streaming_expert_gb300 import sample
    for bad in NO_TENSORS:
        with pytest.raises(ValueError, match="logits"):
            sample(bad, torch.zeros(2))


@pytest.mark.parametrize("rows", [False, True])
def test_pools_that_are_no_tensors(rows):
    from weight_streaming_expert_gb300 import copy_pages, copy_rows
    call = copy_rows if rows else copy_pages
    pool, i = torch.zeros(1, 2, 16, 1, 64), torch.zeros(1, dtype=torch.int64 if rows else torch.int32)
    good = dict(k_pool=pool, v_pool=pool, src=i, dst=i)
    bad_calls(call, good, good)


def test_a_rotation_made_on_the_cpu():
    from weight_streaming_expert_gb300 import QKNormRope
    op, x = QKNormRope(64, device="cpu"), torch.zeros(1, 1, 64).bfloat16()
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CPU"):
        op(x, x, x, None, None, i, i.long(), x[None], x[None])


@pytest.mark.gpu
def test_samples_arguments():
    from weight_streaming_expert_gb300 import sample
    f, i = torch.zeros(2, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    good = dict(logits=torch.zeros(2, 9, device=DEV), u=f, temperature=f, top_k=i, top_p=f, min_p=f, tokens=i)
    bad_calls(sample, good, good, optional=("temperature", "top_k", "top_p", "min_p", "tokens"))
    column = torch.zeros(2, 5, device=DEV)[:, 1:2]
    assert sample(column, f).tolist() == [0, 0]
    with pytest.raises(ValueError, match="top_k"):
        sample(torch.zeros(1, 2, device=DEV).T[:, :1], f, top_k=f)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [False, True])
def test_copies_arguments(rows):
    from weight_streaming_expert_gb300 import copy_pages, copy_rows
    call = copy_rows if rows else copy_pages
    pool = torch.zeros(1, 4, 16, 1, 64, device=DEV)
    i = torch.zeros(1, dtype=torch.int64 if rows else torch.int32, device=DEV)
    good = dict(k_pool=pool, v_pool=pool, src=i, dst=i + 1)
    bad_calls(call, good, good)
    for name in ("src", "dst"):
        with pytest.raises(ValueError, match=name):
            call(**{**good, name: i[0]})


@pytest.mark.gpu
def test_rotations_arguments():
    from weight_streaming_expert_gb300 import QKNormRope
    op = QKNormRope(64, device=DEV)
    x = torch.zeros(2, 2, 64, device=DEV).half()
    cache = torch.zeros(2, 16, 2, 64, device=DEV).half()
    i = torch.zeros(2, dtype=torch.int32, device=DEV)
    good = dict(q=x, k=x, v=x, q_weight=x[0, 0], k_weight=x[0, 0], positions=i, slots=i.long(), k_cache=cache,
                v_cache=cache, q_out=x)
    bad_calls(op, good, good, optional=("q_weight", "k_weight", "q_out"))
    for name in ("q", "k", "k_cache"):
        with pytest.raises(ValueError, match=name):
            op(**{**good, name: x[0, 0, 0]})


@pytest.mark.gpu
def test_attentions_arguments():
    from weight_streaming_expert_gb300 import PagedAttention
    c = Case([2], [40], 4, 2, 64, 16, tree=[1, 3])
    attn = PagedAttention(4, 2, 64, device=DEV)
    good = {**c.inputs(), "out": torch.empty(2, 4, 64, dtype=torch.bfloat16, device=DEV)}
    bad_calls(attn, good, [n for n in good if n not in ("max_q_len", "scale")], optional=("tree_mask", "out"))
    for name in ("max_q_len", "scale"):
        with pytest.raises(ValueError, match=name):
            attn(**{**good, name: "2"})
    for name in ("q", "block_table", "kv_lens"):
        with pytest.raises(ValueError, match=name):
            attn(**{**good, name: good["kv_lens"][0]})
