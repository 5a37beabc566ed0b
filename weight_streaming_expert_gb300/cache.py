"""The paged key/value cache: its memory, its page tables, and the moves of
pages and rows (include/attention.h).  Which sequence holds which page is
decided on the host; the bytes move in the library's kernels."""
from __future__ import annotations

import heapq

import torch

from . import native as N
from .attention import _cache, _elsewhere, _heads, _On, _plain, _scale, _tensor


def _copy(name, rows, k_pool, v_pool, src, dst, stream):
    _tensor("k_pool", k_pool)
    index = k_pool.get_device()
    if index >= 0 and _elsewhere(index, stream):
        with _On(index, stream):
            return _copy(name, rows, k_pool, v_pool, src, dst, None)
    status = N.calls().copy(torch._C._cuda_getCurrentRawStream(index) if index >= 0 else 0, rows, k_pool, v_pool, src,
                            dst)
    if status < 0:
        for n, t in (("v_pool", v_pool), ("src", src), ("dst", dst)):
            _tensor(n, t)
        shape = k_pool.shape
        if len(shape) != 5 or index < 0:
            raise ValueError("the pools must be CUDA tensors [layers, pages, page_size, kv_heads, dim]")
        if v_pool.shape != shape or v_pool.dtype != k_pool.dtype or v_pool.get_device() != index:
            raise ValueError("the pools must have one shape, type and device")
        for n, t in (("src", src), ("dst", dst)):
            _plain(n, t, torch.int64 if rows else torch.int32, index, src.numel())
        raise ValueError("the pools' pages must be contiguous")
    N.check(name, status)


def _scale_pools(k_pool, v_pool, k_scale, v_scale):
    """Looks over the scales [L, P, Hk, page_size] of quantised pools."""
    for name, t, pool_name, pool in (("k_scale", k_scale, "k_pool", k_pool), ("v_scale", v_scale, "v_pool", v_pool)):
        _tensor(name, t)
        _tensor(pool_name, pool)
        if pool.dim() != 5:
            raise ValueError("the pools must be CUDA tensors [layers, pages, page_size, kv_heads, dim]")
        L, P, page_size, heads, _ = pool.shape
        if (t.dtype != torch.uint8 or t.shape != (L, P, heads, page_size) or t.device != pool.device
                or (page_size > 1 and t.stride(3) != 1)):
            raise ValueError(f"{name} must be a uint8 tensor [{L}, {P}, {heads}, {page_size}] with contiguous rows "
                             f"beside {pool_name}")


def copy_pages(k_pool, v_pool, src, dst, stream=None, k_scale=None, v_scale=None):
    """Page dst[i] := page src[i] in every layer of both pools [L, P, page_size,
    Hk, D] (pages contiguous, layers and pages any distance apart); src, dst:
    int32 CUDA tensors [n].  No page may be in dst twice or in both lists.
    k_scale, v_scale [L, P, Hk, page_size] (pages contiguous): those of
    quantised pools, which move too."""
    quantised = k_scale is not None or v_scale is not None
    if quantised:
        _scale_pools(k_pool, v_pool, k_scale, v_scale)
        for t in (k_scale, v_scale):  # before anything has moved
            numbers = (t.shape[2] * t.shape[3], t.stride(0), t.stride(1), t.data_ptr())
            if t.stride(2) != t.shape[3] or any(n % 16 for n in numbers):
                raise ValueError("the scales' pages must be contiguous, of whole 16 bytes, as many apart and aligned to them")
    _copy("moe_copy_pages", False, k_pool, v_pool, src, dst, stream)
    if quantised:
        _copy("moe_copy_pages", False, k_scale.unsqueeze(2), v_scale.unsqueeze(2), src, dst, stream)


def copy_rows(k_pool, v_pool, src, dst, stream=None, k_scale=None, v_scale=None):
    """Cache rows dst[i] := src[i] in every layer of both pools, as if all were
    read before any is written; src, dst: int64 CUDA tensors [n] of slots (page
    * page_size + row), n up to 64, no slot in dst twice.  k_scale, v_scale [L,
    P, Hk, page_size]: those of quantised pools, which move too."""
    quantised = k_scale is not None or v_scale is not None
    if quantised:
        _scale_pools(k_pool, v_pool, k_scale, v_scale)
    _copy("moe_copy_rows", True, k_pool, v_pool, src, dst, stream)
    if quantised:
        index = k_scale.get_device()
        if _elsewhere(index, stream):
            with _On(index, stream):
                return _copy_scales(index, k_scale, v_scale, src, dst)
        _copy_scales(index, k_scale, v_scale, src, dst)


def _copy_scales(index, k_scale, v_scale, src, dst):
    status = N.calls().copy_scales(torch._C._cuda_getCurrentRawStream(index), k_scale, v_scale, src, dst)
    if status < 0:
        raise ValueError("the scales must have one shape and device")
    N.check("moe_copy_scales", status)


def read_cache(k_cache, v_cache, k_scale, v_scale, slots, dtype=torch.bfloat16, k_out=None, v_out=None, stream=None):
    """Rows of one layer of the quantised cache (float8_e4m3fn codes [pages,
    page_size, Hk, D], scales uint8 [pages, Hk, page_size]) as keys and values
    [n, Hk, D] of `dtype`: row i is what lies in slots[i] (int64 [n]), zeros for
    a slot outside the cache.  Exact in bf16."""
    _tensor("k_cache", k_cache)
    index = k_cache.get_device()
    if index >= 0 and _elsewhere(index, stream):
        with _On(index, stream):
            return read_cache(k_cache, v_cache, k_scale, v_scale, slots, dtype, k_out, v_out)
    if dtype not in (torch.bfloat16, torch.float16):
        raise ValueError("dtype must be bf16 or fp16")
    got = N.calls().read_cache(torch._C._cuda_getCurrentRawStream(index) if index >= 0 else 0, dtype == torch.bfloat16,
                               k_cache, v_cache, k_scale, v_scale, slots, k_out, v_out)
    if isinstance(got, int):
        if got < 0:
            if k_cache.dim() != 4 or index < 0:
                raise ValueError("k_cache must be a float8_e4m3fn CUDA tensor [pages, page_size, kv_heads, dim]")
            heads, dim = k_cache.shape[2:]
            for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
                _cache(name, t, torch.float8_e4m3fn, index, heads, dim)
            for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
                _scale(name, t, k_cache, index)
            _tensor("slots", slots)
            _plain("slots", slots, torch.int64, index, slots.numel())
            for name, t in (("k_out", k_out), ("v_out", v_out)):
                if t is not None:
                    _heads(name, t, dtype, index, dim)
            raise ValueError("the caches must have one shape, and the outputs a row for each slot and head")
        N.check("moe_read_e4m3", got)
    return k_out if k_out is not None else got[0], v_out if v_out is not None else got[1]


class PageTable:
    """Which sequence holds which pages (host only; ``PagedKVCache`` moves the
    bytes).  Pages are handed out lowest first and counted: a forked sequence
    shares its parent's full pages."""

    def __init__(self, n_pages: int, page_size: int, max_pages: int):
        if n_pages < 1 or page_size < 1 or max_pages < 1:
            raise ValueError("n_pages, page_size and max_pages must be 1 or more")
        self.n_pages, self.page_size, self.max_pages = n_pages, page_size, max_pages
        self._free = list(range(n_pages))  # a heap: ascending is one
        self._refs = [0] * n_pages
        self._pages: dict[int, list[int]] = {}
        self._lens: dict[int, int] = {}
        self._next = 0

    @property
    def free_pages(self) -> int:
        return len(self._free)

    def sequences(self):
        return list(self._pages)

    def length(self, seq: int) -> int:
        return self._lens[seq]

    def pages(self, seq: int) -> list[int]:
        return list(self._pages[seq])

    def _take(self) -> int:
        page = heapq.heappop(self._free)
        self._refs[page] = 1
        return page

    def _drop(self, page: int):
        self._refs[page] -= 1
        if self._refs[page] == 0:
            heapq.heappush(self._free, page)

    def open(self) -> int:
        """A new, empty sequence."""
        seq, self._next = self._next, self._next + 1
        self._pages[seq], self._lens[seq] = [], 0
        return seq

    def unshare(self, seq: int, start: int, end: int, spare: int = 0):
        """Pages of its own for the positions start..end-1 that lie in shared
        ones, if `spare` more stay free; returns the copies (from, to)."""
        pages, P = self._pages[seq], self.page_size
        last = min(len(pages), -(-end // P)) if start < end else 0
        shared = [i for i in range(start // P, last) if self._refs[pages[i]] > 1]
        if len(shared) + spare > len(self._free):
            raise MemoryError(f"out of pages: {len(self._free)} are free")
        copies = [(pages[i], self._take()) for i in shared]
        for i, (old, new) in zip(shared, copies):
            self._drop(old)
            pages[i] = new
        return copies

    def extend(self, seq: int, n: int):
        """Room for n more positions.  Returns (their slots, page copies (from,
        to) that have to run before they are written: a shared last page)."""
        if n < 0:
            raise ValueError("n must be 0 or more")
        pages, have = self._pages[seq], self._lens[seq]
        need = -(-(have + n) // self.page_size)
        if need > self.max_pages:
            raise ValueError(f"{have + n} positions exceed the {self.max_pages * self.page_size} of a sequence")
        copies = self.unshare(seq, have, have + n, spare=max(0, need - len(pages)))
        while len(pages) < need:
            pages.append(self._take())
        self._lens[seq] = have + n
        P = self.page_size
        return [pages[p // P] * P + p % P for p in range(have, have + n)], copies

    def truncate(self, seq: int, length: int):
        """Keeps the first `length` positions (rejected drafts leave)."""
        if not 0 <= length <= self._lens[seq]:
            raise ValueError(f"length must be in 0..{self._lens[seq]}")
        pages, keep = self._pages[seq], -(-length // self.page_size)
        while len(pages) > keep:
            self._drop(pages.pop())
        self._lens[seq] = length

    def fork(self, seq: int) -> int:
        """A second sequence with the same positions, sharing every page (the
        last one is copied when either of the two writes to it)."""
        new = self.open()
        self._pages[new], self._lens[new] = list(self._pages[seq]), self._lens[seq]
        for page in self._pages[new]:
            self._refs[page] += 1
        return new

    def free(self, seq: int):
        for page in self._pages.pop(seq):
            self._drop(page)
        del self._lens[seq]

    def compact(self):
        """Moves the pages in use to the lowest numbers.  Returns the copies
        (from, to): every `to` was free, so their order is any."""
        used = [p for p in range(self.n_pages) if self._refs[p]]
        holes = [p for p in range(len(used)) if not self._refs[p]]
        moves = dict(zip([p for p in used if p >= len(used)], holes))
        for seq, pages in self._pages.items():
            self._pages[seq] = [moves.get(p, p) for p in pages]
        for a, b in moves.items():
            self._refs[a], self._refs[b] = 0, self._refs[a]
        self._free = list(range(len(used), self.n_pages))
        return list(moves.items())

    def shared_prefix(self, seqs) -> int:
        """How many positions, in whole pages, all of the sequences begin with in
        the same pages and have before their last."""
        first = min((self._pages[s] for s in seqs), key=len, default=[])
        n = 0
        for i, page in enumerate(first):
            if any(self._pages[s][i] != page or self._lens[s] <= (i + 1) * self.page_size for s in seqs):
                break
            n = (i + 1) * self.page_size
        return n

    def slots(self, seq: int, positions):
        P, pages = self.page_size, self._pages[seq]
        return [pages[p // P] * P + p % P for p in positions]


class PagedKVCache:
    """Keys and values of ``n_layers`` layers, ``k`` and ``v`` [L, n_pages,
    page_size, n_kv_heads, head_dim], and the sequences that hold its pages.
    With dtype float8_e4m3fn the cache is quantised: ``k_scale`` and ``v_scale``
    (uint8 [L, n_pages, n_kv_heads, page_size]) hold a power of two for each row
    of a head, else they are None; ``layer(i)`` is what the calls of a layer take.
    It takes half the memory; attention over it is faster than over 16 bits while
    a sequence has few rows for each head of the cache (new tokens times the heads
    that share it): 32 sequences of 2,000 to 32,768 positions take 73 us with 8
    rows (16 bits 131), 91 with 16 (133), 131 with 32 (137), 175 with 64 (124),
    and 415 with 72, which are unpacked first (152).
    The moves run on the current stream (or ``stream``), before what the caller
    enqueues there next."""

    def __init__(self, n_layers: int, n_pages: int, page_size: int, n_kv_heads: int, head_dim: int, max_len: int,
                 dtype=torch.bfloat16, device="cuda"):
        if page_size not in (16, 32, 64, 128, 256):
            raise ValueError("page_size must be 16, 32, 64, 128 or 256")
        shape = (n_layers, n_pages, page_size, n_kv_heads, head_dim)
        self.table = PageTable(n_pages, page_size, -(-max_len // page_size))
        self.k = torch.zeros(shape, dtype=dtype, device=device)
        self.v = torch.zeros(shape, dtype=dtype, device=device)
        self.k_scale = self.v_scale = None
        if dtype == torch.float8_e4m3fn:
            shape = (n_layers, n_pages, n_kv_heads, page_size)
            self.k_scale = torch.full(shape, 127, dtype=torch.uint8, device=device)
            self.v_scale = torch.full(shape, 127, dtype=torch.uint8, device=device)
        self.device = self.k.device

    def layer(self, i: int) -> dict:
        """k_cache and v_cache of a layer, with its scales if it is quantised, as
        named arguments of ``QKNormRope`` and ``PagedAttention``."""
        caches = dict(k_cache=self.k[i], v_cache=self.v[i])
        if self.k_scale is not None:
            caches.update(k_scale=self.k_scale[i], v_scale=self.v_scale[i])
        return caches

    def _device(self, values, dtype, stream):
        t = torch.tensor(values, dtype=dtype)
        if self.device.type != "cuda":
            return t
        with _On(self.device.index, stream):
            return t.pin_memory().to(self.device, non_blocking=True)

    def _copy(self, copies, stream):
        if copies:
            src, dst = self._device(list(zip(*copies)), torch.int32, stream)
            copy_pages(self.k, self.v, src, dst, stream, self.k_scale, self.v_scale)

    def open(self) -> int:
        return self.table.open()

    def length(self, seq: int) -> int:
        return self.table.length(seq)

    def extend(self, seq: int, n: int, stream=None):
        """Room for n more positions; returns their slots, int64 [n] on the
        device.  A last page that a fork shares is copied first."""
        slots, copies = self.table.extend(seq, n)
        self._copy(copies, stream)
        return self._device(slots, torch.int64, stream)

    def truncate(self, seq: int, length: int):
        self.table.truncate(seq, length)

    def fork(self, seq: int) -> int:
        return self.table.fork(seq)

    def free(self, seq: int):
        self.table.free(seq)

    def keep(self, seq: int, start: int, accepted, stream=None):
        """After a verified tree: of the positions start.. only start + i for i
        in `accepted` (ascending) stay, moved up to follow start - 1."""
        accepted = [int(i) for i in accepted]
        if any(b <= a for a, b in zip(accepted, accepted[1:])) or (accepted and accepted[0] < 0):
            raise ValueError("accepted must be ascending positions from 0")
        if not 0 <= start <= self.length(seq) or (accepted and start + accepted[-1] >= self.length(seq)):
            raise ValueError("start + accepted must lie within the sequence")
        moves = [(start + i, start + at) for at, i in enumerate(accepted) if i != at]
        if moves:
            self._copy(self.table.unshare(seq, moves[0][1], moves[-1][1] + 1), stream)
        # blocks in ascending order: what a block writes lies before all that later ones read
        for at in range(0, len(moves), N.MOE_COPY_ROWS_MAX):
            part = moves[at:at + N.MOE_COPY_ROWS_MAX]
            slots = [self.table.slots(seq, at) for at in zip(*part)]
            src, dst = self._device(slots, torch.int64, stream)
            copy_rows(self.k, self.v, src, dst, stream, self.k_scale, self.v_scale)
        self.table.truncate(seq, start + len(accepted))

    def compact(self, stream=None) -> int:
        """Moves the pages in use to the lowest numbers; returns how many moved.
        Block tables made before are stale."""
        moves = self.table.compact()
        self._copy(moves, stream)
        return len(moves)

    def shared_prefix(self, seqs, new: int = 1) -> int:
        """The longest ``prefix_len`` of a ``PagedAttention`` call on the
        sequences (forks) whose last `new` positions each are its new tokens: what
        they begin with in the same whole pages.

        Whether it is worth giving depends on the batch.  With one token and 300
        positions of its own for each sequence (32/4 heads of 128) a call over 16
        bits is faster with a prefix of 4,096 than without from 2 sequences on
        (32: 26 us and 41), with 1,024 about as fast up to 32 and faster with 128
        (44 and 60), with 256 not up to 128; over codes,
        whose pages the sequences find in L2, with 4,096 from somewhere between 32
        and 128 (128: 65 and 82), with 16,384 from 8 or so (26 and 27; 128: 99 and
        246).  Chunks of 64 tokens gain with 4,096 (4 of them 32 and 47), of 512
        and more lose (157 and 131)."""
        page = self.table.page_size
        before = min((self.length(s) for s in seqs), default=0) - new
        return max(0, min(self.table.shared_prefix(seqs), before // page * page))

    def block_table(self, seqs, stream=None):
        """(block table int32 [B, pages of the longest], kv_lens int32 [B]) of
        the sequences, on the device."""
        pages = [self.table.pages(s) for s in seqs]
        width = max([1] + [len(p) for p in pages])
        table = self._device([p + [-1] * (width - len(p)) for p in pages], torch.int32, stream).view(len(pages), width)
        return table, self._device([self.length(s) for s in seqs], torch.int32, stream)
