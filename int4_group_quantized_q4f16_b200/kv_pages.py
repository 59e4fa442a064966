"""Host bookkeeping of a paged KV cache: which pages each sequence holds.

Zero-TVM write-up, section "完整的推理流水线": a paged KV cache read through a
page table.  Sequences may share pages (a forked sequence shares its parent's
full pages); a page that is still being filled belongs to one sequence only, so
appending never writes into a shared page.  Nothing here touches the GPU: the
copies that a fork or a compaction needs are returned as (source, destination)
pages, to be run with ``zt_q4.KvCopy`` before the next append or attention.
"""
from __future__ import annotations

from typing import Dict, Hashable, List, Sequence, Tuple

import numpy as np

Copies = List[Tuple[int, int]]


class KvPages:
    """Pages 0..n_pages-1 of page_size tokens, handed out lowest first."""

    def __init__(self, n_pages: int, page_size: int):
        if n_pages < 1 or page_size < 1:
            raise ValueError("n_pages and page_size must be positive")
        self.n_pages, self.page_size = n_pages, page_size
        self._refs = [0] * n_pages
        self._pages: Dict[Hashable, List[int]] = {}
        self._lens: Dict[Hashable, int] = {}

    def _take(self, n: int) -> List[int]:
        free = [p for p in range(self.n_pages) if not self._refs[p]]
        if n > len(free):
            raise MemoryError(f"{n} pages wanted, {len(free)} of {self.n_pages} free")
        for p in free[:n]:
            self._refs[p] = 1
        return free[:n]

    @property
    def free_pages(self) -> int:
        return self._refs.count(0)

    def sequences(self) -> List[Hashable]:
        return list(self._pages)

    def length(self, seq: Hashable) -> int:
        return self._lens[seq]

    def pages(self, seq: Hashable) -> List[int]:
        return list(self._pages[seq])

    def add(self, seq: Hashable) -> None:
        """A new sequence without tokens."""
        if seq in self._pages:
            raise KeyError(f"sequence {seq!r} exists")
        self._pages[seq], self._lens[seq] = [], 0

    def extend(self, seq: Hashable, tokens: int) -> int:
        """Makes room for `tokens` more tokens; returns the position of the first.  Nothing changes when the pages
        do not suffice (MemoryError)."""
        if tokens < 0:
            raise ValueError("tokens must not be negative")
        start = self._lens[seq]
        want = -(-(start + tokens) // self.page_size) - len(self._pages[seq])
        self._pages[seq] += self._take(max(want, 0))
        self._lens[seq] = start + tokens
        return start

    def fork(self, parent: Hashable, child: Hashable) -> Copies:
        """`child` continues from `parent`'s tokens: full pages are shared, the partly filled last page is copied."""
        if child in self._pages:
            raise KeyError(f"sequence {child!r} exists")
        pages, n = self._pages[parent], self._lens[parent]
        full = n // self.page_size
        own = self._take(len(pages) - full)
        for p in pages[:full]:
            self._refs[p] += 1
        self._pages[child], self._lens[child] = pages[:full] + own, n
        return list(zip(pages[full:], own))

    def free(self, seq: Hashable) -> None:
        """Ends a sequence; pages that no other sequence holds become free."""
        for p in self._pages.pop(seq):
            self._refs[p] -= 1
        del self._lens[seq]

    def compact(self) -> Copies:
        """Moves live pages so that they are pages 0..live-1 (every table changes with them).  Sources and destinations
        are distinct pages, so the copies may run in any order."""
        live = sum(1 for r in self._refs if r)
        moves = dict(zip((p for p in range(live, self.n_pages) if self._refs[p]),
                         (p for p in range(live) if not self._refs[p])))
        for src, dst in moves.items():
            self._refs[dst], self._refs[src] = self._refs[src], 0
        for pages in self._pages.values():
            pages[:] = [moves.get(p, p) for p in pages]
        return list(moves.items())

    def table(self, seqs: Sequence[Hashable], width: int = 0) -> np.ndarray:
        """int32 [len(seqs)][width] page table (width 0: as wide as the longest row, at least 1); unused entries 0."""
        rows = [self._pages[s] for s in seqs]
        width = width or max([1] + [len(r) for r in rows])
        out = np.zeros((len(rows), width), np.int32)
        for i, r in enumerate(rows):
            if len(r) > width:
                raise ValueError(f"sequence {seqs[i]!r} has {len(r)} pages, the table is {width} wide")
            out[i, :len(r)] = r
        return out
