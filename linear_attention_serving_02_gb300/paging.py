"""Which sequence owns which pages of a cache: host logic only.

PagePool counts the references to the pages of one cache (the pages of all layers move
together, so one pool serves them all). Forked sequences share pages until one of them
writes: grow() then asks for a copy of the shared last page. Every method that needs bytes
moved returns the moves as (src, dst) lists for kda.kda_pages_copy, to be made before the
next kernel that writes or reads the pages; the page tables that it hands out are already
the ones after the moves.

A KDA state is one page of a pool with page_size = 1, in a sequence of length 1. It is written
in place at every step, so a copy of a sequence does not share it: add() and grow() the child's
slot, and copy the parent's page there.
"""
import heapq

import torch


class PagePool:
    def __init__(self, num_pages, page_size):
        if num_pages < 0 or page_size <= 0:
            raise ValueError("need num_pages >= 0 and page_size > 0")
        self.num_pages, self.page_size = num_pages, page_size
        self._refs = [0] * num_pages
        self._free = list(range(num_pages))  # a heap: the lowest free page is taken first
        self._pages, self._lens = {}, {}

    @property
    def free_pages(self):
        return len(self._free)

    def sequences(self):
        return list(self._pages)

    def length(self, seq):
        return self._lens[seq]

    def pages(self, seq):
        """The pages of a sequence, in the order of its rows."""
        return list(self._pages[seq])

    def add(self, seq):
        """A new sequence without rows."""
        if seq in self._pages:
            raise ValueError("sequence %r exists" % (seq,))
        self._pages[seq], self._lens[seq] = [], 0

    def fork(self, parent, child):
        """child starts as a copy of parent and shares all its pages; nothing moves yet."""
        if parent not in self._pages:
            raise KeyError(parent)
        self.add(child)
        self._pages[child], self._lens[child] = list(self._pages[parent]), self._lens[parent]
        for p in self._pages[child]:
            self._refs[p] += 1

    def grow(self, seq, tokens):
        """Room for `tokens` more rows of seq. Returns (src, dst): the shared page that they would
        be written into, copied first. Raises MemoryError, and changes nothing, when the pages
        do not suffice."""
        if tokens < 0:
            raise ValueError("tokens must be >= 0")
        pages, length = self._pages[seq], self._lens[seq]
        src, dst = [], []
        shared = tokens > 0 and length % self.page_size != 0 and self._refs[pages[-1]] > 1
        need = -(-(length + tokens) // self.page_size) - len(pages)
        if need + shared > len(self._free):
            raise MemoryError("%d pages are needed and %d are free" % (need + shared, len(self._free)))
        if shared:
            new = self._take()
            src, dst = [pages[-1]], [new]
            self._refs[pages[-1]] -= 1
            pages[-1] = new
        for _ in range(need):
            pages.append(self._take())
        self._lens[seq] = length + tokens
        return src, dst

    def truncate(self, seq, length):
        """Drop the rows of seq from `length` on (rejected draft tokens) and the pages that held them."""
        if not 0 <= length <= self._lens[seq]:
            raise ValueError("length must be between 0 and %d" % self._lens[seq])
        pages, keep = self._pages[seq], -(-length // self.page_size)
        for p in pages[keep:]:
            self._drop(p)
        del pages[keep:]
        self._lens[seq] = length

    def free(self, seq):
        """Give a sequence's pages back; a page shared with another sequence stays that one's."""
        self.truncate(seq, 0)
        del self._pages[seq], self._lens[seq]

    def compact(self):
        """Move the pages in use to the lowest ids. Returns (src, dst); afterwards the pages from
        num_pages - free_pages on are free. Every dst is a page that was free, so the moves
        can run in any order."""
        used = self.num_pages - len(self._free)
        holes = sorted(p for p in self._free if p < used)
        src = [p for p in range(used, self.num_pages) if self._refs[p]]
        to = dict(zip(src, holes))
        for old, new in to.items():
            self._refs[new], self._refs[old] = self._refs[old], 0
        for pages in self._pages.values():
            pages[:] = [to.get(p, p) for p in pages]
        self._free = list(range(used, self.num_pages))
        return src, holes

    def table(self, seqs, max_pages=None):
        """(page_table int32 [N, max_pages], cache_lens int32 [N]) of the sequences, on the CPU; -1
        where a sequence has no page."""
        most = max([len(self._pages[s]) for s in seqs], default=0)
        if max_pages is not None and most > max_pages:
            raise ValueError("a sequence has %d pages, more than max_pages = %d" % (most, max_pages))
        table = torch.full((len(seqs), max(1, most) if max_pages is None else max_pages), -1, dtype=torch.int32)
        for i, s in enumerate(seqs):
            table[i, :len(self._pages[s])] = torch.tensor(self._pages[s], dtype=torch.int32)
        return table, torch.tensor([self._lens[s] for s in seqs], dtype=torch.int32)

    def _take(self):
        p = heapq.heappop(self._free)
        self._refs[p] = 1
        return p

    def _drop(self, p):
        self._refs[p] -= 1
        if self._refs[p] == 0:
            heapq.heappush(self._free, p)
