"""A paged key/value cache whose bookkeeping stays on the device.

One decoding step with drafted trees::

    for layer in range(layers):                      # the target's pass
        ctx = cache.attend(layer, q, k, v, parents, cu_nodes)
    acc, tok, path = sv.spec_verify_tree(...)        # from the pass's probabilities
    cache.commit(k_all, v_all, cu_nodes, acc, path)  # only accepted rows enter

The drafted nodes' keys and values stay outside the cache until they are
accepted; lengths, block tables and the stack of free pages live on the device,
so a step needs nothing from the host.
"""
from __future__ import annotations

import torch

from ._tree import (
    append_args, append_rows, kv_slots, tree_attention, tree_attention_workspace_size,
)


class PagedCache:
    """Keys and values of `batch` requests over `layers` layers: caches
    [layers, pages, page_size, kv_heads, head_dim], a block table for up to
    `max_len` tokens a request.  All calls are made on the current stream (or
    `stream`), one after the other: they share the lengths and one workspace.
    `lens` [batch] holds the cached tokens."""

    def __init__(self, layers: int, pages: int, page_size: int, kv_heads: int, head_dim: int,
                 batch: int, max_len: int, *, dtype=torch.bfloat16, device=None):
        device = torch.device(device or "cuda")
        shape = (layers, pages, page_size, kv_heads, head_dim)
        self.page_size = page_size
        self.k = torch.zeros(shape, dtype=dtype, device=device)
        self.v = torch.zeros(shape, dtype=dtype, device=device)
        width = -(-max_len // page_size)
        self.block_table = torch.full((batch, width), -1, dtype=torch.int32, device=device)
        self.lens = torch.zeros(batch, dtype=torch.int32, device=device)
        # the last entry is taken first: pages are used in increasing order
        self.free_pages = torch.arange(pages - 1, -1, -1, dtype=torch.int32, device=device)
        self.free_count = torch.full((1,), pages, dtype=torch.int32, device=device)
        # one workspace: the calls follow one another (none for layouts attention refuses)
        size = tree_attention_workspace_size(kv_heads, kv_heads, head_dim)
        self._ws = torch.empty(size, dtype=torch.uint8, device=device) if size else None

    def attend(self, layer: int, q, k, v, parents, cu_nodes, *, scale: float | None = None,
               with_lse: bool = False, stream=None):
        """tree_attention of one layer's nodes over this cache: (out, lse)."""
        return tree_attention(q, k, v, self.k[layer], self.v[layer], self.block_table, self.lens,
                              parents, cu_nodes, scale=scale, with_lse=with_lse,
                              workspace=self._ws, stream=stream)

    def extend(self, k, v, cu_rows, add, *, path=None, stream=None):
        """The first add[b] packed rows of every request (or those that `path`
        names) of k, v [layers, N, kv_heads, head_dim] join the cache.  Returns
        start [batch]: the position of the first new token, -1 where there was
        no room (the request stays as it was).  Rows that do not fit the caches
        raise before anything changes."""
        args = append_args(k, v, self.k, self.v)  # refused, if at all, before anything changes
        slots, start, _, _ = kv_slots(self.lens, add, cu_rows, self.block_table, self.free_pages,
                                      self.free_count, rows=k.shape[1], page_size=self.page_size,
                                      path=path, out_lens=self.lens,
                                      out_free_count=self.free_count, stream=stream)
        append_rows(args, slots, k.device, stream)
        return start

    def commit(self, k, v, cu_nodes, accept_len, path=None, *, stream=None):
        """The root and the accepted nodes of a verified step join the cache:
        accept_len and path as spec_verify_tree returns them (path None for
        chains, whose accepted nodes come first).  Sequences that were marked
        (accept_len -1) stay as they were.  Returns start as extend."""
        if stream is None:
            return self.extend(k, v, cu_nodes, accept_len + 1, path=path)
        with torch.cuda.stream(stream):
            return self.extend(k, v, cu_nodes, accept_len + 1, path=path, stream=stream)

    def release(self, which, *, stream=None):
        """The requests with which[b] (bool) give their pages back."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.release(which)
        add = torch.where(which, -1, 0).to(torch.int32)
        none = torch.zeros(which.shape[0] + 1, dtype=torch.int32, device=which.device)
        kv_slots(self.lens, add, none, self.block_table, self.free_pages, self.free_count, rows=0,
                 page_size=self.page_size, out_lens=self.lens, out_free_count=self.free_count)
