"""A paged cache that owns its device buffer through torch and calls libsdv2.

Where :class:`.stream.KVCache` keeps sink frames and a window, this one keeps every token
of its streams, in pages; streams branch off one another without copying what they share,
and the attention reads shared pages once.  torch allocates the buffer and names the stream;
all work runs in the library's kernels (include/sdv2.h, "Paged cache").
"""
from __future__ import annotations

import math

import torch

from . import binding as B
from .prompt import rows_3d

_TORCH = {"bf16": torch.bfloat16, "fp16": torch.float16}


class PagedKVCache:
    """Pages of K and V of ``layers`` layers for up to ``streams`` streams of any length.

    ``counts`` in the calls is one host integer per stream; packed tensors hold the streams'
    tokens in order of the streams.
    """

    def __init__(self, streams, layers, heads, kv_heads, head_dim, pages, page_tokens=64, stream_pages=None,
                 max_queries=None, block_tokens=1, dtype="bf16", device="cuda"):
        if dtype not in _TORCH:
            raise ValueError(f"dtype must be one of {sorted(_TORCH)}, got {dtype!r}")
        self.cfg = B.make_pages_config(streams, layers, heads, kv_heads, head_dim, pages, page_tokens, stream_pages,
                                       max_queries, block_tokens, dtype)
        self.nbytes = B.sdv2_pages_bytes(self.cfg)
        self.handle = None
        self.buffer = torch.empty(self.nbytes, dtype=torch.uint8, device=device)
        if self.buffer.get_device() < 0 or self.buffer.get_device() != B.current_device():
            raise ValueError(f"{self.buffer.device} is not the current device")
        self.device = self.buffer.get_device()
        self.handle = B.sdv2_pages_create(self.cfg, self.buffer, self.nbytes)
        self.layout = B.sdv2_pages_layout_get(self.handle)
        self.streams, self.layers, self.heads, self.kv_heads, self.head_dim = streams, layers, heads, kv_heads, head_dim
        self.pages, self.page_tokens, self.stream_pages = pages, page_tokens, self.cfg.stream_pages
        self.max_queries, self.block_tokens = self.cfg.max_queries, block_tokens
        self.dtype = _TORCH[dtype]
        self._views = {}
        self._any = self.buffer.data_ptr()               # in place of the address that an empty tensor has not
        self._scale = 1.0 / math.sqrt(head_dim)

    def close(self):
        if self.handle:
            B.sdv2_pages_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _counts(self, counts):
        if len(counts) != self.streams:
            raise ValueError(f"counts needs one entry for each of the {self.streams} streams")
        return B.int32_array(counts)

    def _rows(self, x, name, heads, n):
        ptr, stride, tokens = rows_3d(x, name, heads, self.head_dim, self.dtype, self.device)
        if tokens != n:
            raise ValueError(f"{name} has {tokens} tokens, counts say {n}")
        return ptr, stride

    # -- streams and pages
    def extend(self, counts, stream=None):
        """Stream b becomes counts[b] tokens longer (lowest free pages first)."""
        B.sdv2_pages_extend(self.handle, self._counts(counts), stream)

    def fork(self, src, dst, deep=False, stream=None):
        """The empty streams ``dst`` become copies of ``src``, sharing its full pages unless ``deep``."""
        B.sdv2_pages_fork(self.handle, src, dst, deep, stream)

    def free(self, streams, stream=None):
        """The given streams become empty."""
        B.sdv2_pages_free(self.handle, streams, stream)

    def compact(self, stream=None):
        """Moves the used pages to the front of the pool; returns their number."""
        return B.sdv2_pages_compact(self.handle, stream)

    def share(self, mode):
        """When the attention reads pages that forks share once for all: "auto" (where it is faster), "always", "never"."""
        B.sdv2_pages_share(self.handle, mode)

    # -- the path
    def write(self, layer, k, v, counts, stream=None):
        """Keys and values [sum counts, kv_heads, d] of the last counts[b] tokens of each stream."""
        arr = self._counts(counts)
        n = sum(arr)
        kp, ks = self._rows(k, "k", self.kv_heads, n)
        vp, vs = self._rows(v, "v", self.kv_heads, n)
        B.sdv2_pages_write(self.handle, layer, kp or self._any, vp or self._any, ks, vs, arr, stream)

    def attention(self, layer, q, out, counts, softmax_scale=None, stream=None):
        """Queries [sum counts, heads, d] of the last counts[b] tokens of each stream over all its keys."""
        arr = self._counts(counts)
        n = sum(arr)
        qp, qs = self._rows(q, "q", self.heads, n)
        op, os_ = self._rows(out, "out", self.heads, n)
        B.sdv2_pages_attention(self.handle, layer, qp or self._any, op or self._any, qs, os_, arr,
                               self._scale if softmax_scale is None else softmax_scale, stream)

    # -- views of the buffer (for inspection and tests)
    def _region(self, offset, dtype, *shape):
        view = self._views.get((offset, shape))
        if view is None:
            n = math.prod(shape) * dtype.itemsize
            view = self._views[offset, shape] = self.buffer[offset:offset + n].view(dtype).view(*shape)
        return view

    def _pool(self, offset, layer):
        shape = (self.pages, self.kv_heads, self.page_tokens, self.head_dim)
        if layer is None:
            return self._region(offset, self.dtype, self.layers, *shape)
        return self._region(offset + layer * self.layout.layer_stride, self.dtype, *shape)

    def k_pages(self, layer=None):
        """[pages, kv_heads, page_tokens, d] of one layer, or all layers."""
        return self._pool(self.layout.k_offset, layer)

    def v_pages(self, layer=None):
        return self._pool(self.layout.v_offset, layer)

    def page_table(self):
        """int32 [streams, stream_pages]: each stream's pages in order, then -1."""
        return self._region(self.layout.table_offset, torch.int32, self.streams, self.stream_pages)

    def lengths(self):
        """int32 [streams]: tokens of each stream."""
        return self._region(self.layout.length_offset, torch.int32, self.streams)

    def query(self, b):
        """(tokens, page ids, leading pages shared by all streams of b's group), from the host's books."""
        return B.sdv2_pages_query(self.handle, b)

    def used(self):
        return B.sdv2_pages_used(self.handle)

    def check(self):
        return B.sdv2_pages_check(self.handle)
