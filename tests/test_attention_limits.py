"""The limits of an attention call with options, found on the host before
anything is launched."""
import ctypes
import struct

import pytest

from tests.test_attention import args

ROOM = 1 << 62


def forward(heads, prefix, scales=None, workspace=4096, **k):
    """(status, error text) of a call on a handle that holds these numbers alone."""
    from weight_streaming_expert_gb300 import native as N
    L = N.lib()
    # ... and belongs to a device that no machine has: what passes the limits goes no further
    fake = ctypes.create_string_buffer(struct.pack("5i", *heads, 152, 1 << 20), 4096)
    o = N.moe_attn_opts_t(ctypes.pointer(scales) if scales else None, prefix, workspace, ROOM)
    status = L.moe_attn_forward_ex(fake, ctypes.byref(args(**k)), ctypes.byref(o), None)
    return status, N.last_error()


@pytest.mark.parametrize("codes", [False, True])
def test_prefixes_beyond_2_30_positions(codes):
    from weight_streaming_expert_gb300 import native as N
    s = N.moe_cache_scales_t(4096, 4096, 512, 256, 512, 256) if codes else None
    wide = dict(page_size=256, table_stride=1 << 23, n_tokens=1, max_q_len=1)
    for prefix in ((1 << 30) + 256, (1 << 31) - 256):
        status, text = forward((4, 2, 64), prefix, s, **wide)
        assert status == N.MOE_ERR_UNSUPPORTED and "prefix_len" in text, (prefix, text)


def test_limits_count_what_the_lists_do():
    """Items cost three units besides their own, over codes and behind a prefix:
    many short ones are more work than two units each would say."""
    from weight_streaming_expert_gb300 import native as N
    s = N.moe_cache_scales_t(4096, 4096, 1 << 20, 16, 1 << 20, 16)
    heads = (65536, 65536, 64)
    # (32000 / 8 + 4000) items of each head at 1/8 + 1 + 3 units: 2.16e9; at 1/8 + 1 + 2 1.64e9
    status, text = forward(heads, 0, s, batch=4000, n_tokens=32000, max_q_len=1, table_stride=1)
    assert status == N.MOE_ERR_UNSUPPORTED and "too much work" in text, text
    # 4000 * 2 own items at 2/8 + 1 + 3 and 16 over the prefix: 2.23e9 and 1.71e9
    status, text = forward(heads, 16, batch=4000, n_tokens=4000, max_q_len=300, table_stride=2)
    assert status == N.MOE_ERR_UNSUPPORTED and "too much work" in text, text
    # what stays under the limit gets as far as the device
    for prefix, codes in ((0, s), (16, None)):
        status, text = forward(heads, prefix, codes, batch=2000, n_tokens=2000, max_q_len=1, table_stride=2)
        assert status != N.MOE_ERR_UNSUPPORTED, text


@pytest.mark.parametrize("codes", [False, True])
def test_a_longest_chunk_above_all_tokens_is_all_tokens(codes):
    """max_q_len is a bound, and no chunk is longer than the call's tokens: a
    loose one takes no more work or room."""
    from weight_streaming_expert_gb300 import native as N
    L = N.lib()
    s = N.moe_cache_scales_t(4096, 4096, 512, 256, 512, 256) if codes else None
    heads = (8, 2, 64)
    fake = ctypes.create_string_buffer(struct.pack("5i", *heads, 152, 1 << 20), 4096)
    for prefix in (16, 0):
        o = N.moe_attn_opts_t(ctypes.pointer(s) if s else None, prefix, 4096, ROOM)
        room = []
        for longest in (5, 6, 1 << 20, (1 << 31) - 1):
            k = dict(batch=4000, n_tokens=5, max_q_len=longest, table_stride=1 << 10)
            room.append(L.moe_attn_workspace(fake, ctypes.byref(args(**k)), ctypes.byref(o)))
            if s or prefix:
                status, text = forward(heads, prefix, s, **k)
                assert "too much work" not in text and "workspace" not in text, (prefix, longest, text)
        assert room == room[:1] * 4, (prefix, room)


@pytest.mark.gpu
@pytest.mark.parametrize("codes", [False, True])
def test_a_loose_longest_chunk_has_the_same_results(codes):
    import torch

    from tests.test_shared_prefix import Shared
    from weight_streaming_expert_gb300 import PagedAttention
    case = Shared([1, 2, 0, 1], [20, 300, 7, 1], 96, 8, 2, 64, 16, seed=3, codes=codes)
    attn = PagedAttention(8, 2, 64, device="cuda:0")
    x = case.inputs()
    want, want_lse = attn(**{**x, "max_q_len": 4}, return_lse=True)
    case.check(want, want_lse, torch.bfloat16)
    for longest in (1000, 1 << 20, (1 << 31) - 1):
        out, lse = attn(**{**x, "max_q_len": longest}, return_lse=True)
        assert attn.status() == 0 and torch.equal(out, want) and torch.equal(lse, want_lse)
    attn.close()
