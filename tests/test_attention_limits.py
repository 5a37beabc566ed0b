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
