"""Sequences in a 4-bit paged KV cache: which pages hold what, and the calls over them.

    cache = Kv4Cache(n_pages=4096, Hkv=8, d=128, page=64, layers=2)
    a = cache.add()                                  # an empty sequence
    batch = cache.extend([a], [prompt_len])          # room for its next tokens
    for layer in range(2):
        cache.append(layer, k, v, batch)             # K and V rows of those tokens
        o, lse = cache.decode(layer, q, batch)       # attention of the newest Sq tokens
    b = cache.fork(a)                                # shares every page of a
    batch = cache.extend([a, b], [1, 1])             # a part-filled shared page is copied first
    cache.free(a)
    cache.compact()                                  # pages in use moved to the front of the pool

The accounting (free pages, reference counts, page lists) is host arithmetic;
the device work is eio.copy_pages, kv4_append, kv4_read and attn_decode_kv4 on
the current stream.  Use one stream (or order them): a page that is freed may be
written by the next call.  A batch (the page table and lengths of some
sequences, on the device) stays valid until its sequences are extended, freed
or moved by compact(); a call with an older one is refused.
"""
from __future__ import annotations

import heapq

import numpy as np


class Kv4Full(RuntimeError):
    """The pool has too few free pages; the cache is as it was before the call."""


class Kv4Batch:
    """Page table int32 [B,max_pages], lengths int32 [B] and appended counts int32 [B]
    of some sequences of a cache, on its device."""

    def __init__(self, ids, versions, table, seqlens, n_new, most_new):
        self.ids, self.versions = ids, versions
        self.table, self.seqlens, self.n_new, self.most_new = table, seqlens, n_new, most_new


class _Seq:
    __slots__ = ("pages", "length", "version")

    def __init__(self, pages, length, version):
        self.pages, self.length, self.version = pages, length, version


class Kv4Cache:
    """A pool of n_pages pages of `page` tokens for each of `layers` layers, and its sequences."""

    def __init__(self, n_pages, Hkv, d, page=64, layers=1, device=None):
        import torch
        from . import kv4_page_bytes
        if n_pages < 1 or layers < 1:
            raise ValueError(f"n_pages and layers must be >= 1, got {n_pages} and {layers}")
        self.n_pages, self.Hkv, self.d, self.page, self.layers = n_pages, Hkv, d, page, layers
        self.pool = torch.empty((layers, n_pages, Hkv, kv4_page_bytes(page, 1, d)), dtype=torch.uint8,
                                device="cuda" if device is None else device)
        self.device = self.pool.device  # with its number: tables go where the pool is, whatever device is current
        self._refs = np.zeros(n_pages, np.int64)
        self._free = list(range(n_pages))  # a heap: the lowest page first
        self._seqs = {}
        self._next = 0
        self._clock = 0

    # ------------------------------------------------------------ accounting
    def _tick(self):
        self._clock += 1
        return self._clock

    def _seq(self, i):
        if i not in self._seqs:
            raise ValueError(f"no sequence {i} in the cache")
        return self._seqs[i]

    def _drop(self, page):
        self._refs[page] -= 1
        if self._refs[page] == 0:
            heapq.heappush(self._free, page)

    def add(self):
        """A new empty sequence; returns its id."""
        i, self._next = self._next, self._next + 1
        self._seqs[i] = _Seq([], 0, self._tick())
        return i

    def fork(self, i):
        """A new sequence with the tokens of sequence i, in the same pages.  Rows that extend has
        counted but append has not written yet reach both only if they are appended (in every
        layer) before either is extended, which copies a part-filled page as it is."""
        s = self._seq(i)
        for p in s.pages:
            self._refs[p] += 1
        j, self._next = self._next, self._next + 1
        self._seqs[j] = _Seq(list(s.pages), s.length, self._tick())
        return j

    def free(self, i):
        """Forget sequence i; pages that no other sequence holds become free."""
        for p in self._seq(i).pages:
            self._drop(p)
        del self._seqs[i]

    def truncate(self, i, length):
        """Forget the tokens of sequence i at and past `length` (rejected drafts)."""
        s = self._seq(i)
        if not 0 <= length <= s.length:
            raise ValueError(f"length {length} is not within the {s.length} tokens of sequence {i}")
        keep = -(-length // self.page)
        for p in s.pages[keep:]:
            self._drop(p)
        del s.pages[keep:]
        s.length, s.version = length, self._tick()

    def length(self, i):
        return self._seq(i).length

    def free_pages(self):
        return len(self._free)

    def pages_used(self):
        return self.n_pages - len(self._free)

    def _ids(self, ids):
        ids = [int(i) for i in ids]
        if not ids or len(set(ids)) != len(ids):
            raise ValueError(f"a batch needs one or more distinct sequences, got {ids}")
        return ids

    def extend(self, ids, n_new):
        """Make room for n_new (a number, or one for each sequence) more tokens of each of
        the sequences; returns their Kv4Batch, the new tokens counted.  A shared page that
        would be written is copied first.  Raises Kv4Full if the pool has too few free pages.
        Whatever it raises, the cache is as it was before the call."""
        ids = self._ids(ids)
        counts = [int(n_new)] * len(ids) if np.ndim(n_new) == 0 else [int(n) for n in n_new]
        if len(counts) != len(ids) or min(counts) < 0:
            raise ValueError(f"n_new must be one count >= 0 for each of the {len(ids)} sequences, got {n_new}")
        seqs = [self._seq(i) for i in ids]
        need, refs, copies = 0, {}, []
        for s, n in zip(seqs, counts):
            need += -(-(s.length + n) // self.page) - len(s.pages)
            shared = False
            if n and s.length % self.page:  # its last page is written
                p = s.pages[-1]
                refs[p] = refs.get(p, int(self._refs[p])) - 1
                shared = refs[p] >= 1
            need += shared
            copies.append(shared)
        if need > len(self._free):
            raise Kv4Full(f"{need} pages are needed and {len(self._free)} are free")
        # The copies and the upload may fail: pages are only taken until both are done, then the rest changes.
        taken = [heapq.heappop(self._free) for _ in range(need)]
        try:
            src, dst, tails, at = [], [], [], 0  # tails: where a sequence's new pages go in its list, and the pages
            for s, n, shared in zip(seqs, counts, copies):
                first = len(s.pages) - shared
                some = taken[at:at - (-(s.length + n) // self.page) - first]
                at += len(some)
                if shared:
                    src.append(s.pages[-1])
                    dst.append(some[0])
                tails.append((first, some))
            self._copy(src, dst)
            versions = [self._tick() if n else s.version for s, n in zip(seqs, counts)]
            batch = self._batch(ids, counts, versions, tails)
        except BaseException:
            for p in taken:
                heapq.heappush(self._free, p)
            raise
        self._refs[taken] = 1
        for p in src:
            self._refs[p] -= 1
        for s, n, version, (first, some) in zip(seqs, counts, versions, tails):
            if some:
                s.pages[first:] = some
            s.length += n
            s.version = version
        return batch

    def batch(self, ids):
        """The Kv4Batch of sequences as they are (for read or decode)."""
        ids = self._ids(ids)
        seqs = [self._seq(i) for i in ids]
        return self._batch(ids, [0] * len(ids), [s.version for s in seqs], [(len(s.pages), []) for s in seqs])

    def compact(self):
        """Move the pages in use to the front of the pool, so that pages pages_used() ..
        hold nothing.  Returns the number of pages moved; earlier batches become invalid."""
        used = self.pages_used()
        src = [int(p) for p in np.flatnonzero(self._refs[used:]) + used]
        dst = [int(p) for p in np.flatnonzero(self._refs[:used] == 0)]
        if not src:
            return 0
        self._copy(src, dst)
        to = dict(zip(src, dst))
        for s in self._seqs.values():
            s.pages = [to.get(p, p) for p in s.pages]
            s.version = self._tick()
        self._refs[dst] = self._refs[src]
        self._refs[src] = 0
        self._free = list(range(used, self.n_pages))
        return len(src)

    # ------------------------------------------------------------ device work
    def _copy(self, src, dst):
        if src:
            from . import copy_pages
            for layer in range(self.layers):
                copy_pages(self.pool[layer], src, dst)

    def _batch(self, ids, counts, versions, tails):
        """The Kv4Batch of sequences with counts more tokens and with the pages `some` from
        `first` on, as tails gives them."""
        import torch
        seqs = [self._seq(i) for i in ids]
        B, width = len(ids), max(1, max(max(len(s.pages), first + len(some)) for s, (first, some) in zip(seqs, tails)))
        host = np.zeros(B * width + 2 * B, np.int32)  # one copy to the device: table, lengths, counts
        table = host[:B * width].reshape(B, width)
        for b, (s, (first, some)) in enumerate(zip(seqs, tails)):
            table[b, :len(s.pages)] = s.pages
            table[b, first:first + len(some)] = some
        host[B * width:B * width + B] = [s.length + n for s, n in zip(seqs, counts)]
        host[B * width + B:] = counts
        dev = torch.from_numpy(host).to(self.device)
        return Kv4Batch(ids, versions, dev[:B * width].view(B, width), dev[B * width:B * width + B],
                        dev[B * width + B:], max(counts))

    def _current(self, layer, batch):
        if not 0 <= layer < self.layers:
            raise ValueError(f"layer {layer} of a cache of {self.layers} layers")
        if [self._seqs[i].version if i in self._seqs else None for i in batch.ids] != batch.versions:
            raise ValueError("a sequence of this batch was extended, truncated, freed or moved after the batch was made")
        return self.pool[layer]

    def _same_d(self, x, name):
        if x.dim() != 4 or x.shape[3] != self.d:  # the pool's bytes alone would take 64 for 128 and half the page
            raise ValueError(f"{name} has shape {tuple(x.shape)}; the cache holds heads of d = {self.d}")

    def append(self, layer, k, v, batch):
        """Write k, v [B,N,Hkv,d] bf16, row b's first n_new[b] tokens (the rest is padding),
        as the newest tokens of the batch's sequences."""
        from . import kv4_append
        pool = self._current(layer, batch)
        self._same_d(k, "k")
        if k.shape[1] < batch.most_new:
            raise ValueError(f"k has {k.shape[1]} rows a sequence; the batch has up to {batch.most_new} new tokens")
        kv4_append(k, v, pool, batch.table, batch.seqlens, n_new=batch.n_new)

    def read(self, layer, batch, N, start=None):
        """Tokens start[b] .. start[b] + N - 1 of the batch's sequences as bf16 [B,N,Hkv,d]."""
        from . import kv4_read
        return kv4_read(self._current(layer, batch), batch.table, batch.seqlens, N, self.d, start=start)

    def decode(self, layer, q, batch, scale=None, want_lse=True):
        """Attention of the newest Sq tokens, q [B,Sq,Hq,d], over the batch's sequences."""
        from . import attn_decode_kv4
        pool = self._current(layer, batch)
        self._same_d(q, "q")
        return attn_decode_kv4(q, pool, batch.table, batch.seqlens, scale=scale, want_lse=want_lse)
