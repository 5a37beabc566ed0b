"""The paged cache: page tables on the host (CPU tests against a plain list of
what every sequence holds) and the moves of pages and rows on the GPU (exact:
bytes)."""
import random

import pytest
import torch

DEV = "cuda:0"


def check(table, refs=None):
    held = {}
    for s in table.sequences():
        pages = table.pages(s)
        assert len(pages) == -(-table.length(s) // table.page_size) and len(set(pages)) == len(pages)
        for p in pages:
            held[p] = held.get(p, 0) + 1
    assert table.free_pages == table.n_pages - len(held)
    assert held == {p: n for p, n in enumerate(table._refs) if n}
    assert sorted(table._free) == [p for p in range(table.n_pages) if p not in held]


@pytest.mark.parametrize("seed", range(6))
def test_random_histories(seed):
    """Contents written through the slots survive forks, copies on write,
    truncation, freeing and compaction."""
    from weight_streaming_expert_gb300 import PageTable
    rng = random.Random(seed)
    P = rng.choice([1, 2, 16])
    t = PageTable(40, P, 12)
    memory = {}  # slot -> value
    model = {}   # sequence -> its values
    moved = lambda copies: [memory.update({b * P + r: memory[a * P + r]}) for a, b in copies for r in range(P)
                            if a * P + r in memory]
    for step in range(400):
        act = rng.choice(["open", "extend", "extend", "extend", "truncate", "fork", "free", "compact"])
        seqs = list(model)
        if act == "open":
            model[t.open()] = []
        elif act == "compact":
            copies = t.compact()
            sources, targets = [a for a, _ in copies], [b for _, b in copies]
            assert not set(sources) & set(targets) and len(set(targets)) == len(targets)
            moved(copies)
            used = {p for s in t.sequences() for p in t.pages(s)}
            assert used == set(range(len(used)))
        elif seqs:
            s = rng.choice(seqs)
            if act == "extend":
                n = rng.randint(0, 3 * P)
                before = (t.free_pages, t.pages(s), t.length(s))
                try:
                    slots, copies = t.extend(s, n)
                except (MemoryError, ValueError):
                    assert before == (t.free_pages, t.pages(s), t.length(s))
                    continue
                moved(copies)
                for slot in slots:
                    memory[slot] = (step, slot)
                    model[s].append(memory[slot])
            elif act == "truncate":
                n = rng.randint(0, len(model[s]))
                t.truncate(s, n)
                del model[s][n:]
            elif act == "fork" and len(model) < 8:
                model[t.fork(s)] = list(model[s])
            elif act == "free":
                t.free(s)
                del model[s]
        check(t)
        for s, values in model.items():
            assert [memory[i] for i in t.slots(s, range(len(values)))] == values
    for s in list(model):
        t.free(s)
    assert t.free_pages == 40


def test_limits():
    from weight_streaming_expert_gb300 import PageTable
    t = PageTable(3, 16, 2)
    a = t.open()
    with pytest.raises(ValueError):
        t.extend(a, 33)
    with pytest.raises(ValueError):
        t.extend(a, -1)
    t.extend(a, 32)
    b = t.open()
    t.extend(b, 16)
    with pytest.raises(MemoryError):
        t.extend(b, 1)
    with pytest.raises(ValueError):
        t.truncate(b, 17)
    with pytest.raises(KeyError):
        t.free(99)
    for bad in ((0, 16, 1), (1, 0, 1), (1, 16, 0)):
        with pytest.raises(ValueError):
            PageTable(*bad)


def pools(L, n, page, Hk, D, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(L, n, page, Hk, D, generator=g).to(dtype).to(DEV) for _ in range(2)]


@pytest.mark.gpu
@pytest.mark.parametrize("L,n,page,Hk,D,moves", [(1, 2, 16, 1, 64, 1), (3, 9, 16, 2, 128, 4), (42, 6, 64, 4, 128, 1),
                                                 (2, 200, 32, 3, 64, 90), (1, 5, 256, 8, 128, 2), (5, 3, 1, 1, 8, 1)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_copy_pages(L, n, page, Hk, D, moves, dtype):
    from weight_streaming_expert_gb300 import copy_pages
    k, v = pools(L, n, page, Hk, D, dtype)
    order = torch.randperm(n, generator=torch.Generator().manual_seed(n)).to(torch.int32)
    src, dst = order[:moves], order[moves:2 * moves]
    want = [t.clone() for t in (k, v)]
    for t in want:
        t[:, dst.long()] = t[:, src.long()]
    copy_pages(k, v, src.to(DEV), dst.to(DEV))
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])


@pytest.mark.gpu
def test_copy_pages_leaves_out_pages_that_are_not_there():
    from weight_streaming_expert_gb300 import copy_pages
    k, v = pools(2, 8, 16, 2, 64, torch.bfloat16)
    inner = [t[:, 2:6] for t in (k, v)]  # pages of a larger pool
    want = [t.clone() for t in (k, v)]
    for t in want:
        t[:, 2 + 3] = t[:, 2 + 1]
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    copy_pages(*inner, i(-1, 1, 4, 0), i(0, 3, 2, 1 << 30))
    copy_pages(*inner, i(), i())
    torch.cuda.synchronize()
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 2, 7, 63, 64])
@pytest.mark.parametrize("Hk,D", [(1, 64), (4, 128), (3, 64)])
def test_copy_rows_as_if_read_first(n, Hk, D):
    from weight_streaming_expert_gb300 import copy_rows
    k, v = pools(3, 8, 16, Hk, D, torch.float16, seed=n)
    g = torch.Generator().manual_seed(n)
    src, dst = torch.randperm(128, generator=g)[:n], torch.randperm(128, generator=g)[:n]  # they overlap
    want = [t.clone() for t in (k, v)]
    for t, old in zip(want, (k, v)):
        t.view(3, 128, Hk, D)[:, dst] = old.view(3, 128, Hk, D)[:, src]
    copy_rows(k, v, src.to(DEV), dst.to(DEV))
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])


@pytest.mark.gpu
def test_copy_rows_leaves_out_slots_that_are_not_there():
    from weight_streaming_expert_gb300 import copy_rows
    k, v = pools(1, 8, 16, 2, 64, torch.bfloat16)
    inner = [t[:, 2:6] for t in (k, v)]
    want = [t.clone() for t in (k, v)]
    for t in want:
        t[:, 2, 5] = t[:, 5, 15]
    i = lambda *x: torch.tensor(x, dtype=torch.int64, device=DEV)
    copy_rows(*inner, i(-1, 63, 64, 3, 4), i(1, 5, 2, -7, 1 << 40))
    torch.cuda.synchronize()
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(3))
def test_cache_history(seed):
    """A cache's contents through forks, writes, kept rows and compaction,
    against plain lists."""
    from weight_streaming_expert_gb300 import PagedKVCache
    rng = random.Random(seed)
    L, Hk, D, P = 2, 2, 64, 16
    c = PagedKVCache(L, 30, P, Hk, D, max_len=160, dtype=torch.float16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(seed)
    model = {}

    def write(s, n):
        slots = c.extend(s, n)
        rows = torch.randn(L, n, Hk, D, generator=g, device=DEV).half()
        c.k.view(L, -1, Hk, D)[:, slots] = rows
        c.v.view(L, -1, Hk, D)[:, slots] = -rows
        model[s] = torch.cat([model[s], rows], 1)

    for _ in range(60):
        act = rng.choice(["open", "write", "write", "fork", "keep", "free", "compact"])
        if act == "open" and len(model) < 4:
            model[s := c.open()] = torch.empty(L, 0, Hk, D, dtype=torch.float16, device=DEV)
        elif act == "compact":
            c.compact()
        elif model:
            s = rng.choice(list(model))
            room = min(160 - c.length(s), (c.table.free_pages - 1) * P)
            if act == "write" and room > 0:
                write(s, rng.randint(1, min(room, 40)))
            elif act == "fork" and len(model) < 4:
                model[c.fork(s)] = model[s].clone()
            elif act == "keep" and c.length(s) and c.table.free_pages > 2:
                start = rng.randint(max(0, c.length(s) - 12), c.length(s))
                ok = sorted(rng.sample(range(c.length(s) - start), rng.randint(0, c.length(s) - start)))
                c.keep(s, start, ok)
                model[s] = torch.cat([model[s][:, :start], model[s][:, start:][:, ok]], 1)
            elif act == "free":
                c.free(s)
                del model[s]
        for s, want in model.items():
            at = torch.tensor(c.table.slots(s, range(c.length(s))), dtype=torch.int64, device=DEV)
            assert torch.equal(c.k.view(L, -1, Hk, D)[:, at], want)
            assert torch.equal(c.v.view(L, -1, Hk, D)[:, at], -want)
    if model:
        table, lens = c.block_table(list(model))
        for b, s in enumerate(model):
            assert int(lens[b]) == c.length(s)
            assert [p for p in table[b].tolist() if p >= 0] == c.table.pages(s)


def test_refusals():
    import ctypes

    from weight_streaming_expert_gb300 import native as N
    L = N.lib()
    v = lambda x: None if x is None else ctypes.c_void_p(x)

    def pages(k=16, vv=16, layers=2, ls=4096, ps=1024, n_pages=4, size=1024, src=16, dst=16, n=2):
        return L.moe_copy_pages(v(k), v(vv), layers, ls, ls, ps, ps, n_pages, size, v(src), v(dst), n, None)

    def rows(k=16, layers=2, ps=1024, page=16, size=64, src=16, dst=16, n=2):
        return L.moe_copy_rows(v(k), v(16), layers, 4096, 4096, ps, ps, 4, page, size, v(src), v(dst), n, None)

    for bad in (dict(k=None), dict(vv=None), dict(k=8), dict(layers=0), dict(layers=40000), dict(ls=8), dict(ps=1000),
                dict(n_pages=0), dict(size=8), dict(size=0), dict(src=None), dict(dst=2), dict(n=-1)):
        assert pages(**bad) == N.MOE_ERR_INVALID_ARG, bad
        assert N.last_error()
    for bad in (dict(k=None), dict(layers=0), dict(ps=8), dict(page=0), dict(size=24), dict(src=4), dict(dst=None),
                dict(n=-1)):
        assert rows(**bad) == N.MOE_ERR_INVALID_ARG, bad
    assert rows(n=65) == N.MOE_ERR_UNSUPPORTED
    assert pages(n=0) == N.MOE_OK and rows(n=0) == N.MOE_OK


def test_python_refusals():
    from weight_streaming_expert_gb300 import PagedKVCache, copy_pages, copy_rows
    with pytest.raises(ValueError):
        PagedKVCache(1, 4, 24, 1, 64, 100, device="cpu")
    c = PagedKVCache(1, 4, 16, 1, 64, 64, device="cpu")
    s = c.open()
    c.extend(s, 10)
    for start, ok in ((0, [3, 2]), (0, [-1]), (5, [5]), (11, [])):
        with pytest.raises(ValueError):
            c.keep(s, start, ok)
    i = torch.zeros(1, dtype=torch.int32)
    for call in (copy_pages, copy_rows):
        with pytest.raises(ValueError):
            call(c.k, c.v, i, i)  # not on a GPU
