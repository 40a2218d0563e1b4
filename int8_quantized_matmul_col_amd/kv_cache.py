"""A paged key-value cache with its tables on the GPU.

``PagedKVCache`` owns what the ``kv_*`` calls of ``serving`` work on: the pages
of every layer, a table of page ids and a length for each of ``max_seqs``
rows, and a reference count for each page.  A decode step is

    cache.reserve(rows, new_lengths)                     # pages for the new tokens
    for i, layer in enumerate(model):
        cache.append(i, k, v, rows, positions)
        out = cache.attend(i, q, rows)

with nothing copied to the host.  Which row belongs to which request, and
whether the pool has room, is the caller's to know: ``reserve`` and ``fork``
return a status per row on the device.
"""

from __future__ import annotations

from typing import Optional

import torch

from . import serving


class PagedKVCache:
    def __init__(self, num_pages: int, kv_heads: int, head_dim: int, page_size: int = 16,
                 layers: int = 1, max_seqs: int = 1, max_len: Optional[int] = None,
                 dtype=torch.float16, device="cuda"):
        """max_len: the longest sequence a row can hold (default: the pool)."""
        if min(num_pages, kv_heads, head_dim, page_size, layers, max_seqs) < 1:
            raise ValueError("sizes must be positive")
        width = num_pages if max_len is None else (int(max_len) + page_size - 1) // page_size
        shape = (layers, num_pages, kv_heads)
        kw = dict(device=device)
        # rows of a page that no token was written to are never used
        k = torch.empty((*shape, page_size, head_dim), dtype=dtype, **kw)
        v = torch.empty((*shape, head_dim, page_size), dtype=dtype, **kw)
        scales = [torch.empty((*shape, page_size), dtype=torch.float32, **kw)
                  for _ in range(2)] if dtype == torch.int8 else [None, None]
        self.pages = serving.PagedKV(k, v, *scales)
        self.table = torch.full((max_seqs, width), -1, dtype=torch.int32, **kw)
        self.lengths = torch.zeros((max_seqs,), dtype=torch.int32, **kw)
        self.refcount = torch.zeros((num_pages,), dtype=torch.int32, **kw)
        self._layers = [self.pages.layer(i) for i in range(layers)]

    @property
    def page_size(self) -> int:
        return self.pages.page_size

    def layer(self, i: int) -> serving.PagedKV:
        return self._layers[i]

    def reserve(self, rows, new_lengths):
        """kv_pages_reserve: room for new_lengths[i] tokens in row rows[i]."""
        return serving.kv_pages_reserve(self.table, self.lengths, self.refcount, rows, new_lengths,
                                        self.page_size)

    def append(self, layer: int, k, v, rows, positions) -> None:
        """kv_append: token i of k, v to positions[i] of row rows[i]."""
        serving.kv_append(k, v, self._layers[layer], self.table, rows, positions)

    def gather(self, layer: int, rows, positions, dtype=None):
        """kv_gather: the keys and values at these places."""
        return serving.kv_gather(self._layers[layer], self.table, rows, positions, dtype)

    def attend(self, layer: int, q, rows=None, **kw):
        """kv_attention of one new token per row (see there for the options)."""
        return serving.kv_attention(q, self._layers[layer], self.table, self.lengths, rows, **kw)

    def fork(self, parents, children):
        """kv_pages_fork: children[i] becomes a copy of the sequence parents[i]."""
        return serving.kv_pages_fork(self.pages, self.table, self.lengths, self.refcount, parents,
                                     children)

    def free(self, rows) -> None:
        """kv_pages_free: the rows are empty again."""
        serving.kv_pages_free(self.table, self.lengths, self.refcount, rows)

    def compact(self):
        """kv_pages_compact: used pages to the low ids; returns their number
        (int32 [1] on the GPU)."""
        return serving.kv_pages_compact(self.pages, self.table, self.refcount)[2]


__all__ = ["PagedKVCache"]
