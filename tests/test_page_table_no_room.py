"""Room for no further positions asks for nothing: no copy of a shared page, and
no free page."""
from weight_streaming_expert_gb300 import PagedKVCache, PageTable


def test_no_positions_copy_no_page():
    t = PageTable(4, 16, 4)
    a = t.open()
    t.extend(a, 20)
    b = t.fork(a)
    assert t.extend(b, 0) == ([], []) and t.pages(b) == t.pages(a) and t.free_pages == 2
    slots, copies = t.extend(b, 1)
    assert len(slots) == 1 and copies == [(t.pages(a)[1], t.pages(b)[1])]
    assert t.extend(b, 11)[1] == []


def test_no_positions_in_a_full_pool():
    t = PageTable(2, 16, 4)
    a = t.open()
    t.extend(a, 20)
    b = t.fork(a)
    assert t.free_pages == 0
    assert t.extend(b, 0) == ([], []) and t.unshare(b, 20, 20) == []
    c = t.open()
    assert t.extend(c, 0) == ([], []) and t.length(c) == 0


def test_the_cache_too():
    c = PagedKVCache(1, 2, 16, 1, 64, max_len=64, device="cpu")
    a = c.open()
    c.extend(a, 20)
    assert c.extend(c.fork(a), 0).shape == (0,)
