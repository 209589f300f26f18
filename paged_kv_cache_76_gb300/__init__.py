"""Paged-KV-cache attention for NVIDIA GB300 (sm_103a).

The compute path is ``libpa.so`` (hand-written CUDA behind the C ABI of
``include/pa.h``); this package is its ctypes binding:

* :mod:`.ops` - reshape_and_cache, copy_blocks, decode (partial + lse_merge),
  chunked_prefill, device error word; norm_rope_and_cache, verify_tree,
  decode_accumulate, evict_select and compact_kv; a cache held in 4 bits
  (quantize_and_cache, dequantize_kv4, decode_kv4, chunked_prefill_kv4);
  fork_blocks and copy_pages;
* :mod:`.allocator` - the C++ block allocator (free queue, refcounts, share,
  copy-on-write, release behind a compaction);
* :mod:`.build` - compiles the library in-tree.

Importing the package does not load the library; the first call does, and
raises :class:`LibraryMissing` if it has not been built.
"""
from ._lib import LibraryMissing, PAError  # noqa: F401

__version__ = "0.1.0"
