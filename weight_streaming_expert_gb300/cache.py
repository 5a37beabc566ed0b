"""The paged key/value cache: its memory, its page tables, and the moves of
pages and rows (include/attention.h).  Which sequence holds which page is
decided on the host; the bytes move in the library's kernels."""
from __future__ import annotations

import heapq

import torch

from . import native as N
from .attention import _elsewhere, _On, _plain, _tensor


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


def copy_pages(k_pool, v_pool, src, dst, stream=None):
    """Page dst[i] := page src[i] in every layer of both pools [L, P, page_size,
    Hk, D] (pages contiguous, layers and pages any distance apart); src, dst:
    int32 CUDA tensors [n].  No page may be in dst twice or in both lists."""
    _copy("moe_copy_pages", False, k_pool, v_pool, src, dst, stream)


def copy_rows(k_pool, v_pool, src, dst, stream=None):
    """Cache rows dst[i] := src[i] in every layer of both pools, as if all were
    read before any is written; src, dst: int64 CUDA tensors [n] of slots (page
    * page_size + row), n up to 64, no slot in dst twice."""
    _copy("moe_copy_rows", True, k_pool, v_pool, src, dst, stream)


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

    def slots(self, seq: int, positions):
        P, pages = self.page_size, self._pages[seq]
        return [pages[p // P] * P + p % P for p in positions]


class PagedKVCache:
    """Keys and values of ``n_layers`` layers, ``k`` and ``v`` [L, n_pages,
    page_size, n_kv_heads, head_dim], and the sequences that hold its pages.
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
        self.device = self.k.device

    def _device(self, values, dtype, stream):
        t = torch.tensor(values, dtype=dtype)
        if self.device.type != "cuda":
            return t
        with _On(self.device.index, stream):
            return t.pin_memory().to(self.device, non_blocking=True)

    def _copy(self, copies, stream):
        if copies:
            src, dst = self._device(list(zip(*copies)), torch.int32, stream)
            copy_pages(self.k, self.v, src, dst, stream)

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
            copy_rows(self.k, self.v, src, dst, stream)
        self.table.truncate(seq, start + len(accepted))

    def compact(self, stream=None) -> int:
        """Moves the pages in use to the lowest numbers; returns how many moved.
        Block tables made before are stale."""
        moves = self.table.compact()
        self._copy(moves, stream)
        return len(moves)

    def block_table(self, seqs, stream=None):
        """(block table int32 [B, pages of the longest], kv_lens int32 [B]) of
        the sequences, on the device."""
        pages = [self.table.pages(s) for s in seqs]
        width = max([1] + [len(p) for p in pages])
        table = self._device([p + [-1] * (width - len(p)) for p in pages], torch.int32, stream).view(len(pages), width)
        return table, self._device([self.length(s) for s in seqs], torch.int32, stream)
