"""Torch-tensor binding of the paged-KV C ABI (argument marshalling only).

Every function passes ``data_ptr()`` values, sizes and the current CUDA
stream to the function of the same name in ``include/pa.h``; all work runs in
the library's kernels.  Tensors must be contiguous CUDA tensors of the
documented shapes; int32 index tensors live on the same device.  Calls that
take microseconds on the GPU go through the extension of csrc/marshal.cpp when
they are regular, which does the same in a third of the host time.
"""
from __future__ import annotations

import ctypes as C
import functools
import importlib
import math
import threading

import torch

from . import _lib
from ._lib import PA_BF16, PA_FP16, check

__all__ = [
    "reshape_and_cache",
    "copy_blocks",
    "swap_blocks",
    "decode",
    "decode_partial",
    "lse_merge",
    "decode_split_tokens",
    "decode_workspace_size",
    "chunked_prefill",
    "decode_shared_prefix",
    "decode_shared_prefix_workspace_size",
    "decode_shared_prefix_split_tokens",
    "verify_decode",
    "verify_split_tokens",
    "verify_workspace_size",
    "rope_table",
    "norm_rope_and_cache",
    "tree_mask",
    "verify_tree",
    "verify_tree_split_tokens",
    "verify_tree_workspace_size",
    "decode_accumulate",
    "decode_accumulate_split_tokens",
    "decode_accumulate_workspace_size",
    "evict_select",
    "compact_kv",
    "kv4_cache",
    "quantize_and_cache",
    "dequantize_kv4",
    "decode_kv4",
    "decode_kv4_split_tokens",
    "decode_kv4_workspace_size",
    "chunked_prefill_kv4",
    "chunked_prefill_kv4_split_tokens",
    "chunked_prefill_kv4_workspace_size",
    "fork_blocks",
    "copy_pages",
    "get_device_error",
    "selftest_wait_timeout",
    "launch_count",
    "dtype_code",
    "recording",
    "Recording",
]


def dtype_code(dt: torch.dtype) -> int:
    if dt == torch.bfloat16:
        return PA_BF16
    if dt == torch.float16:
        return PA_FP16
    raise TypeError(f"unsupported dtype {dt}: use torch.bfloat16 or torch.float16")


class Recording:
    """Library launches marshalled once, to be issued again as they are.

    Inside ``with recording() as rec:`` the launching functions of this module
    check and marshal their arguments but launch nothing: each appends a
    callable to ``rec.steps`` that issues the same C call with the same
    pointers, sizes and streams.  ``rec.add(fn)`` appends any other step (an
    event record or wait) in order.  ``rec()`` runs the steps in order: the
    same launches for a fraction of the host time of the marshalling (the
    tensors must stay alive and in place).  A recording belongs to the thread
    that opened it; other threads launch as usual meanwhile.
    """

    def __init__(self):
        self.steps = []
        self.keep = []  # tensors a recorded launch writes or reads that the caller did not pass in

    def add(self, fn):
        self.steps.append(fn)

    def __call__(self):
        for fn in self.steps:
            fn()


_tls = threading.local()  # .rec: the open recording of this thread, if any


class recording:
    """Context manager: see :class:`Recording`."""

    def __enter__(self) -> Recording:
        if getattr(_tls, "rec", None) is not None:
            raise RuntimeError("recordings do not nest")
        _tls.rec = Recording()
        return _tls.rec

    def __exit__(self, *exc):
        _tls.rec = None
        return False


# The functions of csrc/marshal.cpp: what they take, they check, allocate and
# launch; None from them means that the call is not of the regular kind, and
# nothing was done.
_SHORT = ("pa_norm_rope_and_cache", "pa_verify_tree_workspace_size", "pa_verify_tree",
          "pa_decode_accumulate_workspace_size", "pa_decode_accumulate", "pa_evict_select", "pa_compact_kv",
          "pa_quantize_and_cache", "pa_dequantize_kv4", "pa_decode_kv4_workspace_size", "pa_decode_kv4",
          "pa_chunked_prefill_kv4_workspace_size", "pa_chunked_prefill_kv4", "pa_fork_blocks_workspace_size",
          "pa_fork_blocks", "pa_copy_pages")
_marshal = None  # the module; False: not built, or for another torch


def _load_marshal():
    global _marshal
    try:
        lib = _lib.lib()
    except _lib.LibraryMissing:  # the long way says so
        return False
    try:
        m = importlib.import_module("._marshal", __package__)
    except ImportError:
        m = None
    # it reads tensors by the layout of the torch it was compiled with
    if getattr(m, "torch_version", None) == str(torch.__version__):
        m.bind(*(C.cast(getattr(lib, name), C.c_void_p).value for name in _SHORT))
        _marshal = m
    else:
        _marshal = False
    return _marshal


def _short_way(stream):
    """May this call go through _marshal?  (A recording wants the marshalled C call.)"""
    if stream is not None or getattr(_tls, "rec", None) is not None:
        return False
    return _marshal if _marshal is not None else _load_marshal()


def _keep(*tensors) -> None:
    """Inside a recording, keep tensors allocated by the call alive with the recording."""
    rec = getattr(_tls, "rec", None)
    if rec is not None:
        rec.keep.extend(t for t in tensors if t is not None)


def _launch(name: str, *args) -> None:
    """Issue (or, inside a recording, record) the C call `name`(*args)."""
    fn = getattr(_lib.lib(), name)
    rec = getattr(_tls, "rec", None)
    if rec is not None:
        rec.add(lambda: check(fn(*args), name))
        return
    check(fn(*args), name)


# the current stream's handle, without the Stream object that
# torch.cuda.current_stream() builds around it (3 us of a call's 15)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream=None):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


def _empty(shape, dtype, device, stream, returned=False):
    """Memory for a launch on `stream` (None: the current one): of that stream's own, since what the current one frees
    or is handed again may be in use there while the launch runs.  `returned`: the caller goes on with it on the
    current stream."""
    if stream is None or device.type != "cuda":
        return torch.empty(shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream(device)
    if stream.cuda_stream == current.cuda_stream:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if returned:
        t.record_stream(current)
    return t


def _dev(t: torch.Tensor, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _i32(t: torch.Tensor, name: str):
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be int32")
    return _dev(t, name)


def _cache_dims(k_cache: torch.Tensor):
    if k_cache.dim() != 4:
        raise ValueError("caches are [num_blocks, block_size, kv_heads, head_dim]")
    return k_cache.shape


# The C calls take raw pointers and sizes; these checks are what keeps a
# mismatched tensor from being read as the wrong type, past its end, or from
# another GPU's memory.
def _check_caches(k_cache, v_cache):
    _cache_dims(k_cache)
    if v_cache.shape != k_cache.shape or v_cache.dtype != k_cache.dtype or v_cache.device != k_cache.device:
        raise ValueError("k_cache and v_cache must agree in shape, dtype and device")


def _check_index(ref, name: str, t, rows: int, cols: int = None, table: bool = False):
    """An index tensor on ref's device with `rows` leading entries; 2-D with
    `cols` columns if given, 2-D if `table`."""
    if t.device != ref.device:
        raise ValueError(f"{name} is on {t.device}, not {ref.device}")
    two_d = table or cols is not None
    if t.dim() == 0 or t.shape[0] != rows or (two_d and t.dim() != 2) or (cols is not None and t.shape[1] != cols):
        raise ValueError(f"{name} has shape {tuple(t.shape)}: {rows} rows{' x ' + str(cols) if cols else ''} expected")


def _check_attention(q, k_cache, v_cache, out):
    """q, both caches and out share one dtype and device; out has q's shape."""
    _check_caches(k_cache, v_cache)
    if k_cache.dtype != q.dtype or out.dtype != q.dtype:
        raise TypeError(f"q ({q.dtype}), the caches ({k_cache.dtype}) and out ({out.dtype}) must share a dtype")
    if k_cache.device != q.device or out.device != q.device:
        raise ValueError("q, the caches and out must be on one device")
    if out.shape != q.shape:
        raise ValueError(f"out has shape {tuple(out.shape)}, q {tuple(q.shape)}")


def launch_count() -> int:
    return int(_lib.lib().pa_launch_count())


def reshape_and_cache(k, v, slot_mapping, k_cache, v_cache, stream=None):
    nb, bs, hkv, d = _cache_dims(k_cache)
    _check_caches(k_cache, v_cache)
    if k.shape != v.shape or k.dim() != 3 or k.shape[1:] != (hkv, d):
        raise ValueError("k and v are [num_tokens, kv_heads, head_dim] of the cache")
    if k.dtype != k_cache.dtype or v.dtype != k_cache.dtype or k.device != k_cache.device or v.device != k.device:
        raise ValueError("k and v must have the cache's dtype and device")
    _check_index(k, "slot_mapping", slot_mapping, int(k.shape[0]))
    _launch(
        "pa_reshape_and_cache",
        _dev(k, "k"), _dev(v, "v"), _i32(slot_mapping, "slot_mapping"), int(k.shape[0]),
        _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"), nb, bs, hkv, d, dtype_code(k_cache.dtype),
        _stream(stream))


def copy_blocks(k_cache, v_cache, pairs, stream=None):
    """``pairs``: int32 [n, 2] (src, dst) on the cache's device."""
    nb, bs, hkv, d = _cache_dims(k_cache)
    _check_caches(k_cache, v_cache)
    _check_index(k_cache, "pairs", pairs, int(pairs.shape[0]) if pairs.dim() else -1, 2)
    _launch(
        "pa_copy_blocks",
        _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"), _i32(pairs, "pairs"), int(pairs.shape[0]),
        nb, bs, hkv, d, dtype_code(k_cache.dtype), _stream(stream))


def _dev_or_pinned(t: torch.Tensor, name: str):
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if not (t.is_cuda or t.is_pinned()):
        raise ValueError(f"{name} must be a CUDA tensor or pinned host memory")
    return t.data_ptr()


def swap_blocks(src_k, src_v, dst_k, dst_v, pairs, stream=None):
    """Copy blocks between two pools of the cache layout, either of which may
    live in pinned host memory (``pin_memory=True``); ``pairs``: int32 [n, 2]
    (src, dst), on the device or pinned.  Asynchronous on ``stream``."""
    if src_v.shape != src_k.shape or dst_v.shape != dst_k.shape or src_k.shape[1:] != dst_k.shape[1:] \
            or src_k.dtype != dst_k.dtype or src_v.dtype != src_k.dtype or dst_v.dtype != dst_k.dtype:
        raise ValueError("the pools must agree in block shape and dtype")
    if pairs.dtype != torch.int32:
        raise TypeError("pairs must be int32")
    ns, bs, hkv, d = _cache_dims(src_k)
    nd = dst_k.shape[0]
    _launch(
        "pa_swap_blocks",
        _dev_or_pinned(src_k, "src_k"), _dev_or_pinned(src_v, "src_v"), _dev_or_pinned(dst_k, "dst_k"),
        _dev_or_pinned(dst_v, "dst_v"), _dev_or_pinned(pairs, "pairs"), int(pairs.shape[0]), ns, nd, bs, hkv, d,
        dtype_code(src_k.dtype), _stream(stream))


def decode_split_tokens(max_blocks_per_seq: int, block_size: int, split_tokens: int = 0) -> int:
    return check(_lib.lib().pa_decode_split_tokens(max_blocks_per_seq, block_size, split_tokens),
                 "pa_decode_split_tokens")


def decode_workspace_size(num_seqs, q_heads, head_dim, max_blocks_per_seq, block_size, split_tokens=0) -> int:
    return int(_lib.lib().pa_decode_workspace_size(num_seqs, q_heads, head_dim, max_blocks_per_seq,
                                                   block_size, split_tokens))


def _check_decode(q, k_cache, v_cache, block_tables, context_lens, out):
    nb, bs, hkv, d = _cache_dims(k_cache)
    if q.dim() != 3 or q.shape[2] != d:
        raise ValueError("q is [num_seqs, q_heads, head_dim] of the cache's head_dim")
    _check_attention(q, k_cache, v_cache, out)
    _check_index(q, "block_tables", block_tables, int(q.shape[0]), table=True)
    _check_index(q, "context_lens", context_lens, int(q.shape[0]))


def _decode_args(q, k_cache, v_cache, block_tables, context_lens, scale, out, split_tokens, workspace):
    nb, bs, hkv, d = _cache_dims(k_cache)
    B, hq, dq = q.shape
    _check_decode(q, k_cache, v_cache, block_tables, context_lens, out)
    maxblk = int(block_tables.shape[1])
    ws_ptr, ws_bytes = (workspace.data_ptr(), workspace.numel() * workspace.element_size()) \
        if workspace is not None else (None, 0)
    return (_dev(q, "q"), _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"), _i32(block_tables, "block_tables"),
            maxblk, _i32(context_lens, "context_lens"), B, hq, hkv, d, bs, nb, float(scale), int(split_tokens),
            ws_ptr, ws_bytes, _dev(out, "out"), dtype_code(q.dtype))


def make_workspace(q, block_tables, block_size, split_tokens=0, stream=None):
    """Allocate (with torch) the scratch that :func:`decode` needs, or None."""
    B, hq, d = q.shape
    n = decode_workspace_size(B, hq, d, int(block_tables.shape[1]), block_size, split_tokens)
    if n == 0:
        return None
    return _empty(n, torch.uint8, q.device, stream)


def decode(q, k_cache, v_cache, block_tables, context_lens, scale, out=None, split_tokens=0, workspace=None,
           stream=None):
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream, returned=True)
    _check_decode(q, k_cache, v_cache, block_tables, context_lens, out)
    if workspace is None:
        workspace = make_workspace(q, block_tables, k_cache.shape[1], split_tokens, stream)
    args = _decode_args(q, k_cache, v_cache, block_tables, context_lens, scale, out, split_tokens, workspace)
    _keep(out, workspace)
    _launch("pa_decode", *args, _stream(stream))
    return out


def decode_partial(q, k_cache, v_cache, block_tables, context_lens, scale, out, split_tokens=0, workspace=None,
                   stream=None):
    args = _decode_args(q, k_cache, v_cache, block_tables, context_lens, scale, out, split_tokens, workspace)
    _launch("pa_decode_partial", *args, _stream(stream))


def lse_merge(workspace, context_lens, q, block_tables, block_size, out, split_tokens=0, stream=None):
    B, hq, d = q.shape
    if out.shape != q.shape or out.device != q.device:
        raise ValueError("out must have q's shape and device")
    _check_index(q, "context_lens", context_lens, B)
    ws_ptr, ws_bytes = (workspace.data_ptr(), workspace.numel() * workspace.element_size()) \
        if workspace is not None else (None, 0)
    _launch("pa_lse_merge", ws_ptr, ws_bytes, _i32(context_lens, "context_lens"), B, hq, d,
            int(block_tables.shape[1]), block_size, int(split_tokens), _dev(out, "out"), dtype_code(out.dtype),
            _stream(stream))


def verify_split_tokens(max_blocks_per_seq: int, block_size: int, q_len: int, split_tokens: int = 0) -> int:
    return check(_lib.lib().pa_verify_split_tokens(max_blocks_per_seq, block_size, q_len, split_tokens),
                 "pa_verify_split_tokens")


def verify_workspace_size(num_seqs, q_len, q_heads, head_dim, max_blocks_per_seq, block_size, split_tokens=0) -> int:
    return int(_lib.lib().pa_verify_workspace_size(num_seqs, q_len, q_heads, head_dim, max_blocks_per_seq,
                                                   block_size, split_tokens))


def verify_decode(q, k_cache, v_cache, block_tables, context_lens, scale, out=None, split_tokens=0, workspace=None,
                  stream=None):
    """pa_verify_decode: ``q`` is [num_seqs, k+1, q_heads, head_dim]; query i of
    request r sees its first ``context_lens[r] - k + i`` tokens."""
    nb, bs, hkv, d = _cache_dims(k_cache)
    if q.dim() != 4:
        raise ValueError("q is [num_seqs, q_len, q_heads, head_dim]")
    B, ql, hq, dq = q.shape
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream, returned=True)
    if dq != d:
        raise ValueError("head_dim mismatch")
    _check_attention(q, k_cache, v_cache, out)
    _check_index(q, "block_tables", block_tables, B, table=True)
    _check_index(q, "context_lens", context_lens, B)
    maxblk = int(block_tables.shape[1])
    if workspace is None:
        n = verify_workspace_size(B, ql, hq, d, maxblk, bs, split_tokens)
        workspace = _empty(n, torch.uint8, q.device, stream) if n else None
    ws_ptr, ws_bytes = (workspace.data_ptr(), workspace.numel() * workspace.element_size()) \
        if workspace is not None else (None, 0)
    _keep(out, workspace)
    _launch(
        "pa_verify_decode",
        _dev(q, "q"), _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"), _i32(block_tables, "block_tables"), maxblk,
        _i32(context_lens, "context_lens"), B, ql, hq, hkv, d, bs, nb, float(scale), int(split_tokens), ws_ptr,
        ws_bytes, _dev(out, "out"), dtype_code(q.dtype), _stream(stream))
    return out


def decode_shared_prefix_workspace_size(num_seqs, q_heads, head_dim, max_blocks_per_seq, block_size, prefix_len,
                                        split_tokens=0) -> int:
    return int(_lib.lib().pa_decode_shared_prefix_workspace_size(num_seqs, q_heads, head_dim, max_blocks_per_seq,
                                                                 block_size, prefix_len, split_tokens))


def decode_shared_prefix_split_tokens(max_blocks_per_seq, block_size, prefix_len, split_tokens=0) -> int:
    """Suffix partition size pa_decode_shared_prefix uses (0: its automatic choice)."""
    return check(_lib.lib().pa_decode_shared_prefix_split_tokens(int(max_blocks_per_seq), int(block_size),
                                                                 int(prefix_len), int(split_tokens)),
                 "pa_decode_shared_prefix_split_tokens")


def decode_shared_prefix(q, k_cache, v_cache, prefix_blocks, prefix_len, block_tables, context_lens, scale, out=None,
                         split_tokens=0, workspace=None, stream=None, prefix_stream=None):
    """pa_decode_shared_prefix: decode whose requests share ``prefix_blocks`` (int32, device).

    ``prefix_stream`` (a torch.cuda.Stream): run the prefix pass there,
    concurrently with the suffix pass; the caller orders it after the writes
    of ``q``, the prefix's K/V and the previous use of ``workspace`` (None:
    after all that is under way on ``stream``, whose memory it is)."""
    nb, bs, hkv, d = _cache_dims(k_cache)
    B, hq, dq = q.shape
    if dq != d:
        raise ValueError("head_dim mismatch")
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream, returned=True)
    _check_attention(q, k_cache, v_cache, out)
    _check_index(q, "block_tables", block_tables, B, table=True)
    _check_index(q, "context_lens", context_lens, B)
    if prefix_blocks.device != q.device or prefix_blocks.numel() < int(prefix_len) // bs:
        raise ValueError("prefix_blocks must hold prefix_len / block_size block ids on q's device")
    maxblk = int(block_tables.shape[1])
    if workspace is None:
        n = decode_shared_prefix_workspace_size(B, hq, d, maxblk, bs, int(prefix_len), split_tokens)
        workspace = _empty(max(n, 1), torch.uint8, q.device, stream)
    _keep(out, workspace)
    _launch(
        "pa_decode_shared_prefix",
        _dev(q, "q"), _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"), _i32(prefix_blocks, "prefix_blocks"),
        int(prefix_len), _i32(block_tables, "block_tables"), maxblk, _i32(context_lens, "context_lens"), B, hq, hkv,
        d, bs, nb, float(scale), int(split_tokens), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _dev(out, "out"),
        dtype_code(q.dtype), _stream(stream), prefix_stream.cuda_stream if prefix_stream is not None else None)
    return out


def verify_decode_tc(q, k_cache, v_cache, block_tables, context_lens, scale, out=None, max_ctas=0, stream=None):
    """pa_verify_decode_tc: ``q`` is [num_seqs, k+1, q_heads, head_dim]; the
    verify attention on the tcgen05 kernel (no workspace)."""
    nb, bs, hkv, d = _cache_dims(k_cache)
    B, ql, hq, dq = q.shape
    if dq != d:
        raise ValueError("head_dim mismatch")
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream, returned=True)
    _check_attention(q, k_cache, v_cache, out)
    _check_index(q, "block_tables", block_tables, B, table=True)
    _check_index(q, "context_lens", context_lens, B)
    _keep(out)
    _launch("pa_verify_decode_tc", _dev(q, "q"), _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"),
            _i32(block_tables, "block_tables"), int(block_tables.shape[1]), _i32(context_lens, "context_lens"), B,
            ql, hq, hkv, d, bs, nb, float(scale), int(max_ctas), _dev(out, "out"), dtype_code(q.dtype),
            _stream(stream))
    return out


def chunked_prefill(q, q_start, context_lens, k_cache, v_cache, block_tables, scale, max_q_len, out=None,
                    stream=None, max_ctas=0):
    """pa_chunked_prefill; ``max_ctas`` > 0 caps the CTAs (SMs) the tensor-core path uses."""
    nb, bs, hkv, d = _cache_dims(k_cache)
    T, hq, dq = q.shape
    if dq != d:
        raise ValueError("head_dim mismatch")
    R = int(context_lens.shape[0])
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream, returned=True)
    _check_attention(q, k_cache, v_cache, out)
    _check_index(q, "context_lens", context_lens, R)
    _check_index(q, "q_start", q_start, R + 1)
    _check_index(q, "block_tables", block_tables, R, table=True)
    _keep(out)
    _launch(
        "pa_chunked_prefill",
        _dev(q, "q"), _i32(q_start, "q_start"), _i32(context_lens, "context_lens"), _dev(k_cache, "k_cache"),
        _dev(v_cache, "v_cache"), _i32(block_tables, "block_tables"), int(block_tables.shape[1]), R, T,
        int(max_q_len), int(max_ctas), hq, hkv, d, bs, nb, float(scale), _dev(out, "out"), dtype_code(q.dtype),
        _stream(stream))
    return out


# The calls below take microseconds on the GPU, so their checks are written for
# few interpreter steps: a device is its index (-1: not a GPU's), a tensor is
# checked and its pointer taken in one place, and pure functions of sizes are
# remembered.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _stream_on(dev: int, stream=None):
    """The launch's stream; the library launches on the current device, where every tensor has to be."""
    if dev < 0:
        raise ValueError("the tensors must be CUDA tensors")
    if dev != _current_device():
        raise ValueError(f"the tensors are on cuda:{dev}, but the current device is cuda:{_current_device()}")
    if stream is not None:
        return stream.cuda_stream
    return _raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream().cuda_stream


def _ptr(t: torch.Tensor, name: str, dev: int) -> int:
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not with the other tensors")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows_ptr(t: torch.Tensor, name: str, dev: int, rows: int) -> int:
    """An int32 index tensor with `rows` leading entries."""
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be int32")
    shape = t.shape
    if not shape or shape[0] != rows:
        raise ValueError(f"{name} has shape {tuple(shape)}: {rows} rows expected")
    return _ptr(t, name, dev)


def _table_ptr(t: torch.Tensor, dev: int, rows: int) -> int:
    if t.dim() != 2:
        raise ValueError("block_tables is [num_seqs, max_blocks_per_seq]")
    return _rows_ptr(t, "block_tables", dev, rows)


def _cache_ptrs(k_cache, v_cache, dev: int):
    """(k, v) pointers of two caches of one shape and dtype."""
    if k_cache.dim() != 4:
        raise ValueError("caches are [num_blocks, block_size, kv_heads, head_dim]")
    if v_cache.shape != k_cache.shape or v_cache.dtype != k_cache.dtype:
        raise ValueError("k_cache and v_cache must agree in shape, dtype and device")
    return _ptr(k_cache, "k_cache", dev), _ptr(v_cache, "v_cache", dev)


def _score_ptrs(scores, hkv: int, score_rows, num_seqs: int, dev: int, name="scores"):
    """(scores, score_rows) pointers."""
    shape = scores.shape
    if len(shape) != 3 or shape[1] != hkv or scores.dtype != torch.float32:
        raise ValueError(f"{name} is fp32 [rows, kv_heads, length]")
    if score_rows is not None:
        return _ptr(scores, name, dev), _rows_ptr(score_rows, "score_rows", dev, num_seqs)
    if shape[0] < num_seqs:
        raise ValueError(f"{name} has fewer rows than there are requests")
    return _ptr(scores, name, dev), None


def rope_table(max_position: int, rot_dim: int, base: float = 10000.0, device=None) -> torch.Tensor:
    """fp32 [max_position, rot_dim], cosines then sines of ``position * base^(-2j/rot_dim)``: the table
    :func:`norm_rope_and_cache` reads.  The angles are taken in 64 bits: in 32 those of far positions lose the
    digits that matter."""
    j = torch.arange(rot_dim // 2, dtype=torch.float64, device=device)
    angle = torch.arange(max_position, dtype=torch.float64, device=device)[:, None] * base ** (-2.0 * j / rot_dim)
    return torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32)


def _token_rows(t: torch.Tensor, name: str, heads: int, d: int, dtype, dev: int) -> int:
    """Token stride (elements) of [num_tokens, heads, head_dim] whose heads are contiguous."""
    if t.dtype != dtype:
        raise TypeError(f"{name} ({t.dtype}) must have the cache's dtype ({dtype})")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not with the other tensors")
    row = heads * d
    if t.is_contiguous():
        stride = row
    else:
        s0, s1, s2 = t.stride()
        if s2 != 1 or (heads > 1 and s1 != d):
            raise ValueError(f"{name}: the heads of a token must be contiguous")
        stride = s0 if t.shape[0] > 1 else row
    if stride < row or stride & 7:
        raise ValueError(f"{name}: tokens must be at least a row, and a multiple of 8 elements, apart")
    return stride


@functools.lru_cache(maxsize=256)
def _sections(counts):
    """(the C array, the counts' sum, the smallest)"""
    return (C.c_int32 * 3)(*counts), sum(counts), min(counts)


def norm_rope_and_cache(q, k, v, positions, cos_sin, slot_mapping, k_cache, v_cache, q_weight=None, k_weight=None,
                        eps=1e-6, sections=None, interleaved=False, out=None, stream=None):
    """pa_norm_rope_and_cache: per-head norm (with ``q_weight``/``k_weight``) and rotary position of new queries and
    keys, keys and values into their slots; returns the queries.

    ``q``/``k``/``v`` may be views of one projection's rows.  ``positions``: int32 [num_tokens], or
    [axes, num_tokens] with ``sections`` (pairs per axis).  ``out`` may be ``q`` if that is contiguous."""
    if _short_way(stream):
        r = _marshal.norm_rope(q, k, v, positions, cos_sin, slot_mapping, k_cache, v_cache, q_weight, k_weight, eps,
                               sections, interleaved, out)
        if r is not None:
            if type(r) is int:
                check(r, "pa_norm_rope_and_cache")
            return r
    dtype, dev = k_cache.dtype, k_cache.get_device()
    kc, vc = _cache_ptrs(k_cache, v_cache, dev)
    nb, bs, hkv, d = k_cache.shape
    if q.dim() != 3 or q.shape[2] != d:
        raise ValueError("q is [num_tokens, q_heads, head_dim] of the cache's head_dim")
    qshape = T, hq, _ = q.shape
    if k.shape != (T, hkv, d) or v.shape != (T, hkv, d):
        raise ValueError("k and v are [num_tokens, kv_heads, head_dim] of the cache, as many tokens as q")
    qs = _token_rows(q, "q", hq, d, dtype, dev)
    ks = _token_rows(k, "k", hkv, d, dtype, dev)
    vs = _token_rows(v, "v", hkv, d, dtype, dev)
    pshape = positions.shape
    axes = 1 if len(pshape) == 1 else pshape[0] if len(pshape) == 2 else 0
    if not 1 <= axes <= 3 or pshape[-1] != T:
        raise ValueError("positions is [num_tokens] or [1 to 3 axes, num_tokens]")
    if cos_sin.dim() != 2 or cos_sin.dtype != torch.float32:
        raise ValueError("cos_sin is fp32 [max_position, rot_dim]")
    max_pos, rot = cos_sin.shape
    sec = None
    if sections is None:
        if axes > 1:
            raise ValueError("several axes need their sections")
    else:
        sec, pairs, least = _sections(tuple(sections)) if len(sections) == axes else (None, -1, -1)
        if least < 0 or pairs != rot // 2:
            raise ValueError(f"sections are {axes} counts of pairs, rot_dim / 2 = {rot // 2} together")
    qw = kw = None
    if q_weight is not None:
        if q_weight.shape != (d,) or q_weight.dtype != dtype:
            raise ValueError("q_weight is [head_dim] of q's dtype")
        qw = _ptr(q_weight, "q_weight", dev)
    if k_weight is not None:
        if k_weight.shape != (d,) or k_weight.dtype != dtype:
            raise ValueError("k_weight is [head_dim] of q's dtype")
        kw = _ptr(k_weight, "k_weight", dev)
    sl = _rows_ptr(slot_mapping, "slot_mapping", dev, T)
    if out is None:
        out = _empty(qshape, dtype, q.device, stream, returned=True)
    elif out.shape != qshape or out.dtype != dtype:
        raise ValueError("out must have q's shape, dtype and device")
    handle = _stream_on(dev, stream)
    _keep(out)
    _launch(
        "pa_norm_rope_and_cache", q.data_ptr(), k.data_ptr(), v.data_ptr(), qs, ks, vs, qw, kw, eps,
        _rows_ptr(positions, "positions", dev, pshape[0]), axes, sec, _ptr(cos_sin, "cos_sin", dev), max_pos, rot,
        1 if interleaved else 0, sl, T, hq, _ptr(out, "out", dev), kc, vc, nb, bs, hkv, d, dtype_code(dtype), handle)
    return out


def tree_mask(parents) -> torch.Tensor:
    """int64 [n] (host): node i sees itself and its ancestors.  ``parents[i]`` < i, or -1 for a child of the context."""
    words = []
    for i, p in enumerate(parents):
        p = int(p)
        if not -1 <= p < i or i >= 64:
            raise ValueError("parents come before their children, at most 64 nodes")
        words.append((words[p] if p >= 0 else 0) | 1 << i)
    return torch.tensor([w - (1 << 64) if w >> 63 else w for w in words], dtype=torch.int64)


def verify_tree_split_tokens(num_reqs, max_q_len, q_heads, kv_heads, max_blocks_per_seq, block_size,
                             split_tokens=0) -> int:
    return check(_lib.lib().pa_verify_tree_split_tokens(int(num_reqs), int(max_q_len), int(q_heads), int(kv_heads),
                                                        int(max_blocks_per_seq), int(block_size), int(split_tokens)),
                 "pa_verify_tree_split_tokens")


def verify_tree_workspace_size(num_reqs, total_q, max_q_len, q_heads, kv_heads, head_dim, max_blocks_per_seq,
                               block_size, split_tokens=0) -> int:
    return int(_lib.lib().pa_verify_tree_workspace_size(num_reqs, total_q, max_q_len, q_heads, kv_heads, head_dim,
                                                        max_blocks_per_seq, block_size, split_tokens))


@functools.lru_cache(maxsize=4096)
def _tree_workspace(dev, *sizes) -> int:  # dev: the choice depends on the current device
    return verify_tree_workspace_size(*sizes)


def verify_tree(q, q_start, tree_mask, context_lens, k_cache, v_cache, block_tables, scale, max_q_len, out=None,
                split_tokens=0, workspace=None, stream=None):
    """pa_verify_tree: ``q`` is [total_q, q_heads, head_dim], packed by ``q_start``; bit m of ``tree_mask[i]`` (int64)
    lets row i see its request's node m.  Every row sees the context before the draft.  ``scale`` is positive.
    ``split_tokens`` 0 runs large batches whole: give one (16384, say) where a context is far longer than the rest."""
    if workspace is None and _short_way(stream):
        r = _marshal.verify_tree(q, q_start, tree_mask, context_lens, k_cache, v_cache, block_tables, scale, max_q_len,
                                 out, split_tokens)
        if r is not None:
            if type(r) is int:
                check(r, "pa_verify_tree")
            return r
    dtype, dev = q.dtype, q.get_device()
    kc, vc = _cache_ptrs(k_cache, v_cache, dev)
    nb, bs, hkv, d = k_cache.shape
    if q.dim() != 3 or q.shape[2] != d:
        raise ValueError("q is [total_q, q_heads, head_dim] of the cache's head_dim")
    qshape = T, hq, _ = q.shape
    if k_cache.dtype != dtype or (out is not None and out.dtype != dtype):
        raise TypeError(f"q ({dtype}), the caches ({k_cache.dtype}) and out must share a dtype")
    R = context_lens.shape[0]
    lens = _rows_ptr(context_lens, "context_lens", dev, R)
    starts = _rows_ptr(q_start, "q_start", dev, R + 1)
    tables = _table_ptr(block_tables, dev, R)
    if tree_mask.dtype != torch.int64:
        raise TypeError("tree_mask must be int64")
    if tree_mask.dim() == 0 or tree_mask.shape[0] != T:
        raise ValueError(f"tree_mask has shape {tuple(tree_mask.shape)}: {T} rows expected")
    mask = _ptr(tree_mask, "tree_mask", dev)
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream, returned=True)
    elif out.shape != qshape:
        raise ValueError(f"out has shape {tuple(out.shape)}, q {tuple(qshape)}")
    handle = _stream_on(dev, stream)
    maxblk = block_tables.shape[1]
    max_q_len, split_tokens = int(max_q_len), int(split_tokens)
    if workspace is None:
        n = _tree_workspace(dev, R, T, max_q_len, hq, hkv, d, maxblk, bs, split_tokens)
        workspace = _empty(n, torch.uint8, q.device, stream) if n else None
    ws_ptr, ws_bytes = (_ptr(workspace, "workspace", dev), workspace.numel() * workspace.element_size()) \
        if workspace is not None else (None, 0)
    _keep(out, workspace)
    _launch(
        "pa_verify_tree", _ptr(q, "q", dev), starts, mask, lens, kc, vc, tables, maxblk, R, T, max_q_len, hq, hkv, d,
        bs, nb, float(scale), split_tokens, ws_ptr, ws_bytes, _ptr(out, "out", dev), dtype_code(dtype), handle)
    return out


def decode_accumulate_split_tokens(num_seqs, q_heads, kv_heads, max_blocks_per_seq, block_size, split_tokens=0) -> int:
    """Partition size such a pa_decode_accumulate call uses (0: its automatic choice)."""
    return check(_lib.lib().pa_decode_accumulate_split_tokens(int(num_seqs), int(q_heads), int(kv_heads),
                                                              int(max_blocks_per_seq), int(block_size),
                                                              int(split_tokens)), "pa_decode_accumulate_split_tokens")


def decode_accumulate_workspace_size(num_seqs, q_heads, kv_heads, head_dim, max_blocks_per_seq, block_size,
                                     split_tokens=0) -> int:
    return int(_lib.lib().pa_decode_accumulate_workspace_size(num_seqs, q_heads, kv_heads, head_dim,
                                                              max_blocks_per_seq, block_size, split_tokens))


@functools.lru_cache(maxsize=4096)
def _accumulate_workspace(dev, *sizes) -> int:  # dev: the choice depends on the current device
    return decode_accumulate_workspace_size(*sizes)


def decode_accumulate(q, k_cache, v_cache, block_tables, context_lens, scale, scores, score_rows=None,
                      scores_out=None, out=None, split_tokens=0, workspace=None, stream=None):
    """pa_decode_accumulate: :func:`decode`, and each cached token's attention weight (summed over the query heads of
    its KV head) added to its score.  ``scores``: fp32 [rows, kv_heads, length], request r's row is ``score_rows[r]``
    (None: r; negative: no score).  ``scores_out`` None: in place.  Returns (out, scores_out).

    Prompts and drafts keep no score: only this call's queries do.  The scratch and the second pass grow with the
    width of ``block_tables``, so cut them to the longest context."""
    if workspace is None and _short_way(stream):
        r = _marshal.decode_accumulate(q, k_cache, v_cache, block_tables, context_lens, scale, scores, score_rows,
                                       scores_out, out, split_tokens)
        if r is not None:
            if type(r) is int:
                check(r, "pa_decode_accumulate")
            return r
    dtype, dev = q.dtype, q.get_device()
    kc, vc = _cache_ptrs(k_cache, v_cache, dev)
    nb, bs, hkv, d = k_cache.shape
    if q.dim() != 3 or q.shape[2] != d:
        raise ValueError("q is [num_seqs, q_heads, head_dim] of the cache's head_dim")
    qshape = B, hq, _ = q.shape
    if k_cache.dtype != dtype or (out is not None and out.dtype != dtype):
        raise TypeError(f"q ({dtype}), the caches ({k_cache.dtype}) and out must share a dtype")
    tables = _table_ptr(block_tables, dev, B)
    lens = _rows_ptr(context_lens, "context_lens", dev, B)
    sc, rows = _score_ptrs(scores, hkv, score_rows, B, dev)
    so = sc
    if scores_out is None:
        scores_out = scores
    else:
        if scores_out.shape != scores.shape:
            raise ValueError("scores_out must have scores' shape")
        so, _ = _score_ptrs(scores_out, hkv, None, 0, dev, "scores_out")
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream, returned=True)
    elif out.shape != qshape:
        raise ValueError(f"out has shape {tuple(out.shape)}, q {tuple(qshape)}")
    handle = _stream_on(dev, stream)
    maxblk, split_tokens = block_tables.shape[1], int(split_tokens)
    if workspace is None:
        n = _accumulate_workspace(dev, B, hq, hkv, d, maxblk, bs, split_tokens)
        workspace = _empty(max(n, 1), torch.uint8, q.device, stream)
    _keep(out, workspace)
    _launch(
        "pa_decode_accumulate", _ptr(q, "q", dev), kc, vc, tables, maxblk, lens, B, hq, hkv, d, bs, nb, float(scale),
        split_tokens, sc, rows, scores.shape[0], scores.shape[2], so, _ptr(workspace, "workspace", dev),
        workspace.numel() * workspace.element_size(), _ptr(out, "out", dev), dtype_code(dtype), handle)
    return out, scores_out


def evict_select(scores, context_lens, sink, heavy, recent, score_rows=None, keep=None, keep_lens=None, stream=None):
    """pa_evict_select: per request and KV head the tokens a budget of ``sink + heavy + recent`` keeps, ascending:
    the first, the last, and the best scored between.  Returns (keep int32 [num_seqs, kv_heads, budget], -1 behind;
    keep_lens int32 [num_seqs]); neither may be an input's memory (``context_lens`` among them)."""
    if keep is None and keep_lens is None and _short_way(stream):
        r = _marshal.evict_select(scores, context_lens, sink, heavy, recent, score_rows)
        if r is not None:
            if type(r) is int:
                check(r, "pa_evict_select")
            return r
    if scores.dim() != 3:
        raise ValueError("scores is fp32 [rows, kv_heads, length]")
    dev = scores.get_device()
    nrows, hkv, length = scores.shape
    B = context_lens.shape[0]
    lens = _rows_ptr(context_lens, "context_lens", dev, B)
    sc, rows = _score_ptrs(scores, hkv, score_rows, B, dev)
    sink, heavy, recent = int(sink), int(heavy), int(recent)
    budget = sink + heavy + recent
    if sink < 0 or heavy < 0 or recent < 0 or budget < 1:
        raise ValueError("sink, heavy and recent are counts, at least one token together")
    if keep is None:
        keep = _empty((B, hkv, budget), torch.int32, scores.device, stream, returned=True)
    elif keep.shape != (B, hkv, budget):
        raise ValueError(f"keep is int32 [{B}, {hkv}, {budget}]")
    if keep_lens is None:
        keep_lens = _empty(B, torch.int32, scores.device, stream, returned=True)
    handle = _stream_on(dev, stream)
    _keep(keep, keep_lens)
    _launch(
        "pa_evict_select", sc, rows, nrows, hkv, length, lens, B, sink, heavy, recent,
        _rows_ptr(keep, "keep", dev, B), _rows_ptr(keep_lens, "keep_lens", dev, B), handle)
    return keep, keep_lens


def compact_kv(k_cache, v_cache, block_tables, context_lens, keep, keep_lens, base=None, scores=None, score_rows=None,
               stream=None):
    """pa_compact_kv: token ``base[r] + i`` of each sequence becomes its token ``base[r] + keep[r, g, i]``, in place
    (``keep``: int32 [num_seqs, 1 or kv_heads, max_keep], ``i <= keep[i]``); with ``scores``, those too, and zeros
    behind them."""
    if _short_way(stream):
        r = _marshal.compact_kv(k_cache, v_cache, block_tables, context_lens, keep, keep_lens, base, scores, score_rows)
        if r is not None:
            check(r, "pa_compact_kv")
            return
    dev = k_cache.get_device()
    kc, vc = _cache_ptrs(k_cache, v_cache, dev)
    nb, bs, hkv, d = k_cache.shape
    B = context_lens.shape[0]
    tables = _table_ptr(block_tables, dev, B)
    lens = _rows_ptr(context_lens, "context_lens", dev, B)
    kshape = keep.shape
    if len(kshape) != 3 or kshape[1] not in (1, hkv):
        raise ValueError("keep is int32 [num_seqs, 1 or kv_heads, max_keep]")
    lists = _rows_ptr(keep, "keep", dev, B)
    nkeep = _rows_ptr(keep_lens, "keep_lens", dev, B)
    first = _rows_ptr(base, "base", dev, B) if base is not None else None
    sc = rows = None
    nrows = length = 0
    if scores is not None:
        sc, rows = _score_ptrs(scores, hkv, score_rows, B, dev)
        nrows, _, length = scores.shape
    handle = _stream_on(dev, stream)
    if kshape[2] == 0:
        if scores is not None:
            raise ValueError("keep has no entries")
        return
    _launch(
        "pa_compact_kv", kc, vc, tables, block_tables.shape[1], lens, lists, kshape[1], kshape[2], nkeep, first, B, nb,
        bs, hkv, d, dtype_code(k_cache.dtype), sc, rows, nrows, length, handle)


# ----------------------------------------------------------------------------
# a cache held in 4 bits
# ----------------------------------------------------------------------------
def kv4_cache(num_blocks, block_size, kv_heads, head_dim, device="cuda"):
    """A cache of 4-bit elements, uint8 [num_blocks, kv_heads, block_size * head_dim * 9 / 16], all zeros: one of K or
    of V.  The calls find block_size from its shape and the head_dim of the 16-bit tensors."""
    if block_size not in (4, 8, 16, 32) or head_dim not in (64, 128):
        raise ValueError("block_size is 4, 8, 16 or 32, head_dim 64 or 128")
    return torch.zeros((num_blocks, kv_heads, block_size * head_dim * 9 // 16), dtype=torch.uint8, device=device)


def _kv4_ptrs(k_cache, v_cache, dev: int, d: int):
    """(k, v) pointers of two 4-bit caches and their (num_blocks, block_size, kv_heads)."""
    shape = k_cache.shape
    if len(shape) != 3 or k_cache.dtype != torch.uint8:
        raise ValueError("4-bit caches are uint8 [num_blocks, kv_heads, page bytes]")
    if v_cache.shape != shape or v_cache.dtype != torch.uint8:
        raise ValueError("k_cache and v_cache must agree in shape, dtype and device")
    bs, rest = divmod(shape[2] * 16, 9 * d) if d > 0 else (0, 1)
    if rest or bs not in (4, 8, 16, 32):
        raise ValueError(f"pages of {shape[2]} bytes are not those of blocks of 4, 8, 16 or 32 tokens of head_dim {d}")
    return _ptr(k_cache, "k_cache", dev), _ptr(v_cache, "v_cache", dev), shape[0], bs, shape[1]


def quantize_and_cache(k, v, slot_mapping, k_cache, v_cache, stream=None):
    """pa_quantize_and_cache: :func:`reshape_and_cache` into a 4-bit cache.  ``k`` and ``v`` ([num_tokens, kv_heads,
    head_dim]) may be views of one projection's rows."""
    if _short_way(stream):
        r = _marshal.quantize_and_cache(k, v, slot_mapping, k_cache, v_cache)
        if r is not None:
            check(r, "pa_quantize_and_cache")
            return
    if k.dim() != 3 or v.shape != k.shape:
        raise ValueError("k and v are [num_tokens, kv_heads, head_dim] of the cache")
    dtype, dev = k.dtype, k.get_device()
    T, hkv, d = k.shape
    kc, vc, nb, bs, heads = _kv4_ptrs(k_cache, v_cache, dev, d)
    if heads != hkv:
        raise ValueError(f"the caches have {heads} heads, k and v {hkv}")
    code = dtype_code(dtype)
    ks = _token_rows(k, "k", hkv, d, dtype, dev)
    vs = _token_rows(v, "v", hkv, d, dtype, dev)
    sl = _rows_ptr(slot_mapping, "slot_mapping", dev, T)
    _launch("pa_quantize_and_cache", k.data_ptr(), v.data_ptr(), ks, vs, sl, T, kc, vc, nb, bs, hkv, d, code,
            _stream_on(dev, stream))


def dequantize_kv4(k_cache, v_cache, slots, head_dim, dtype=torch.bfloat16, k=None, v=None, stream=None):
    """pa_dequantize_kv4: K and V of the tokens at ``slots`` in 16 bits, each [num_tokens, kv_heads, head_dim] (exact;
    zeros where a slot is negative).  Small outputs share one allocation."""
    if k is None and v is None and _short_way(stream):
        r = _marshal.dequantize_kv4(k_cache, v_cache, slots, head_dim, dtype_code(dtype))
        if r is not None:
            if type(r) is int:
                check(r, "pa_dequantize_kv4")
            return r
    dev, d, code = k_cache.get_device(), int(head_dim), dtype_code(dtype)
    kc, vc, nb, bs, hkv = _kv4_ptrs(k_cache, v_cache, dev, d)
    T = slots.shape[0] if slots.dim() == 1 else -1
    sl = _rows_ptr(slots, "slots", dev, T)
    handle = _stream_on(dev, stream)
    shape = (T, hkv, d)
    out = []
    for name, t in (("k", k), ("v", v)):
        if t is None:
            t = _empty(shape, dtype, k_cache.device, stream, returned=True)
        elif t.shape != shape or t.dtype != dtype:
            raise ValueError(f"{name} is {dtype} {list(shape)}")
        out.append(t)
    _keep(*out)
    _launch("pa_dequantize_kv4", kc, vc, sl, T, nb, bs, hkv, d, _ptr(out[0], "k", dev), _ptr(out[1], "v", dev), code,
            handle)
    return tuple(out)


def decode_kv4_split_tokens(num_seqs, q_len, q_heads, kv_heads, max_blocks_per_seq, block_size, split_tokens=0) -> int:
    """Partition size such a pa_decode_kv4 call uses (0: its automatic choice)."""
    return check(_lib.lib().pa_decode_kv4_split_tokens(int(num_seqs), int(q_len), int(q_heads), int(kv_heads),
                                                       int(max_blocks_per_seq), int(block_size), int(split_tokens)),
                 "pa_decode_kv4_split_tokens")


def decode_kv4_workspace_size(num_seqs, q_len, q_heads, kv_heads, head_dim, max_blocks_per_seq, block_size,
                              split_tokens=0) -> int:
    return int(_lib.lib().pa_decode_kv4_workspace_size(num_seqs, q_len, q_heads, kv_heads, head_dim,
                                                       max_blocks_per_seq, block_size, split_tokens))


@functools.lru_cache(maxsize=4096)
def _kv4_workspace(dev, *sizes) -> int:  # dev: the choice depends on the current device
    return decode_kv4_workspace_size(*sizes)


def _scratch(workspace, n: int, device, dev: int, stream):
    """(the workspace, its pointer and bytes): the caller's, or one of n bytes."""
    if workspace is None:
        if not n:
            return None, None, 0
        workspace = _empty(n, torch.uint8, device, stream)
    return workspace, _ptr(workspace, "workspace", dev), workspace.numel() * workspace.element_size()


def decode_kv4(q, k_cache, v_cache, block_tables, context_lens, scale, out=None, split_tokens=0, workspace=None,
               stream=None):
    """pa_decode_kv4: :func:`decode` (``q`` [num_seqs, q_heads, head_dim]) or :func:`verify_decode` (``q`` [num_seqs,
    q_len, q_heads, head_dim]) over a 4-bit cache."""
    if workspace is None and _short_way(stream):
        r = _marshal.decode_kv4(q, k_cache, v_cache, block_tables, context_lens, scale, out, split_tokens)
        if r is not None:
            if type(r) is int:
                check(r, "pa_decode_kv4")
            return r
    if q.dim() not in (3, 4):
        raise ValueError("q is [num_seqs, q_heads, head_dim] or [num_seqs, q_len, q_heads, head_dim]")
    dtype, dev, qshape = q.dtype, q.get_device(), q.shape
    B, ql, hq, d = (qshape[0], 1, qshape[1], qshape[2]) if len(qshape) == 3 else qshape
    kc, vc, nb, bs, hkv = _kv4_ptrs(k_cache, v_cache, dev, d)
    code = dtype_code(dtype)
    tables = _table_ptr(block_tables, dev, B)
    lens = _rows_ptr(context_lens, "context_lens", dev, B)
    if out is None:
        out = _empty(qshape, dtype, q.device, stream, returned=True)
    elif out.shape != qshape or out.dtype != dtype:
        raise ValueError("out must have q's shape, dtype and device")
    handle = _stream_on(dev, stream)
    maxblk, split_tokens = block_tables.shape[1], int(split_tokens)
    n = _kv4_workspace(dev, B, ql, hq, hkv, d, maxblk, bs, split_tokens) if workspace is None else 0
    workspace, ws_ptr, ws_bytes = _scratch(workspace, n, q.device, dev, stream)
    _keep(out, workspace)
    _launch("pa_decode_kv4", _ptr(q, "q", dev), kc, vc, tables, maxblk, lens, B, ql, hq, hkv, d, bs, nb, float(scale),
            split_tokens, ws_ptr, ws_bytes, _ptr(out, "out", dev), code, handle)
    return out


def chunked_prefill_kv4_split_tokens(num_reqs, max_q_len, q_heads, kv_heads, max_blocks_per_seq, block_size,
                                     split_tokens=0) -> int:
    """Partition size such a pa_chunked_prefill_kv4 call uses (0: its automatic choice)."""
    return check(_lib.lib().pa_chunked_prefill_kv4_split_tokens(int(num_reqs), int(max_q_len), int(q_heads),
                                                                int(kv_heads), int(max_blocks_per_seq),
                                                                int(block_size), int(split_tokens)),
                 "pa_chunked_prefill_kv4_split_tokens")


def chunked_prefill_kv4_workspace_size(num_reqs, total_q, max_q_len, q_heads, kv_heads, head_dim, max_blocks_per_seq,
                                       block_size, split_tokens=0) -> int:
    return int(_lib.lib().pa_chunked_prefill_kv4_workspace_size(num_reqs, total_q, max_q_len, q_heads, kv_heads,
                                                                head_dim, max_blocks_per_seq, block_size,
                                                                split_tokens))


@functools.lru_cache(maxsize=4096)
def _kv4_prefill_workspace(dev, *sizes) -> int:  # dev: the choice depends on the current device
    return chunked_prefill_kv4_workspace_size(*sizes)


def chunked_prefill_kv4(q, q_start, context_lens, k_cache, v_cache, block_tables, scale, max_q_len, out=None,
                        split_tokens=0, workspace=None, stream=None):
    """pa_chunked_prefill_kv4: :func:`chunked_prefill` over a 4-bit cache.  ``scale`` is not zero."""
    if workspace is None and _short_way(stream):
        r = _marshal.chunked_prefill_kv4(q, q_start, context_lens, k_cache, v_cache, block_tables, scale, max_q_len, out,
                                         split_tokens)
        if r is not None:
            if type(r) is int:
                check(r, "pa_chunked_prefill_kv4")
            return r
    if q.dim() != 3:
        raise ValueError("q is [total_q, q_heads, head_dim]")
    dtype, dev, qshape = q.dtype, q.get_device(), q.shape
    T, hq, d = qshape
    kc, vc, nb, bs, hkv = _kv4_ptrs(k_cache, v_cache, dev, d)
    code = dtype_code(dtype)
    R = context_lens.shape[0]
    lens = _rows_ptr(context_lens, "context_lens", dev, R)
    starts = _rows_ptr(q_start, "q_start", dev, R + 1)
    tables = _table_ptr(block_tables, dev, R)
    if out is None:
        out = _empty(qshape, dtype, q.device, stream, returned=True)
    elif out.shape != qshape or out.dtype != dtype:
        raise ValueError("out must have q's shape, dtype and device")
    handle = _stream_on(dev, stream)
    maxblk, max_q_len, split_tokens = block_tables.shape[1], int(max_q_len), int(split_tokens)
    n = _kv4_prefill_workspace(dev, R, T, max_q_len, hq, hkv, d, maxblk, bs, split_tokens) if workspace is None else 0
    workspace, ws_ptr, ws_bytes = _scratch(workspace, n, q.device, dev, stream)
    _keep(out, workspace)
    _launch("pa_chunked_prefill_kv4", _ptr(q, "q", dev), starts, lens, kc, vc, tables, maxblk, R, T, max_q_len, hq, hkv,
            d, bs, nb, float(scale), split_tokens, ws_ptr, ws_bytes, _ptr(out, "out", dev), code, handle)
    return out


# ----------------------------------------------------------------------------
# sequences that go on from others
# ----------------------------------------------------------------------------
@functools.lru_cache(maxsize=4096)
def _fork_workspace(dev, num_new, num_blocks) -> int:  # dev: the size depends on the current device
    return int(_lib.lib().pa_fork_blocks_workspace_size(num_new, num_blocks))


def fork_blocks(block_tables, context_lens, parents, num_blocks, block_size, grow=1, max_grow=None, pinned=None,
                max_blocks=None, workspace=None, stream=None):
    """pa_fork_blocks: new row i goes on from row ``parents[i]`` (-1: a new sequence, below: none) and grows by ``grow``
    tokens (a count, or int32 [num_new] of at most ``max_grow``).  Returns (tables int32 [num_new, max_blocks], lens
    [num_new], pairs [num_new, 2] for :func:`copy_pages`, slots [num_new, max_grow], num_free [1]).

    ``pinned`` (bool or uint8 [num_blocks]): blocks that others hold.  ``max_blocks``: columns of the new tables (None:
    as many as ``block_tables`` has).  The outputs may share one allocation."""
    if workspace is None and _short_way(stream):
        r = _marshal.fork_blocks(block_tables, context_lens, parents, num_blocks, block_size, grow, max_grow, pinned,
                                 max_blocks)
        if r is not None:
            if type(r) is int:
                check(r, "pa_fork_blocks")
            return r
    dev, num_blocks, block_size = block_tables.get_device(), int(num_blocks), int(block_size)
    B, R = context_lens.shape[0], parents.shape[0]
    tables = _table_ptr(block_tables, dev, B)
    lens = _rows_ptr(context_lens, "context_lens", dev, B)
    par = _rows_ptr(parents, "parents", dev, R)
    gr = pin = None
    if isinstance(grow, torch.Tensor):
        if max_grow is None:
            raise ValueError("a tensor of growths needs max_grow")
        gr = _rows_ptr(grow, "grow", dev, R)
        max_grow = int(max_grow)
    else:
        if max_grow is not None and int(max_grow) != int(grow):
            raise ValueError("max_grow is for a tensor of growths")
        max_grow = int(grow)
    if max_grow < 0:
        raise ValueError("growths are counts")
    if pinned is not None:
        if pinned.dtype not in (torch.bool, torch.uint8) or pinned.shape != (num_blocks,):
            raise ValueError("pinned is bool or uint8 [num_blocks]")
        pin = _ptr(pinned, "pinned", dev)
    handle = _stream_on(dev, stream)
    width = block_tables.shape[1] if max_blocks is None else int(max_blocks)
    if width < 1:
        raise ValueError("the new tables have no columns")

    def new(*shape):
        return _empty(shape, torch.int32, block_tables.device, stream, returned=True)
    out = (new(R, width), new(R), new(R, 2), new(R, max_grow), new(1))
    n = _fork_workspace(dev, R, num_blocks) if workspace is None else 0
    workspace, ws_ptr, ws_bytes = _scratch(workspace, n, block_tables.device, dev, stream)
    _keep(*out, workspace)
    _launch("pa_fork_blocks", tables, block_tables.shape[1], lens, B, par, R, gr, max_grow, pin, num_blocks, block_size,
            out[0].data_ptr(), width, out[1].data_ptr(), out[2].data_ptr(), out[3].data_ptr(), out[4].data_ptr(), ws_ptr,
            ws_bytes, handle)
    return out


def copy_pages(caches, pairs, stream=None):
    """pa_copy_pages: in every cache (a list of tensors [num_blocks, ...] of one size, 16-bit or 4-bit) block
    ``pairs[p, 1]`` becomes a copy of block ``pairs[p, 0]``; a negative source is no copy."""
    if _short_way(stream):
        r = _marshal.copy_pages(caches, pairs)
        if r is not None:
            check(r, "pa_copy_pages")
            return
    caches = list(caches)
    if not caches:
        return
    dev = caches[0].get_device()
    nb = caches[0].shape[0] if caches[0].dim() else 0
    size = caches[0].numel() * caches[0].element_size()
    ptrs = []
    for i, c in enumerate(caches):
        if not c.dim() or c.shape[0] != nb or c.numel() * c.element_size() != size:
            raise ValueError("the caches must agree in blocks and bytes")
        ptrs.append(_ptr(c, f"caches[{i}]", dev))
    if not nb or size // nb % 16:
        raise ValueError("a block is a multiple of 16 bytes")
    if pairs.dim() != 2 or pairs.shape[1] != 2:
        raise ValueError("pairs is int32 [num_pairs, 2]")
    pr = _rows_ptr(pairs, "pairs", dev, pairs.shape[0])
    _launch("pa_copy_pages", (C.c_void_p * len(ptrs))(*ptrs), len(ptrs), pr, pairs.shape[0], nb, size // nb,
            _stream_on(dev, stream))


def selftest_wait_timeout(wait_ms: int = 50, stream=None) -> None:
    """Launch the library's bounded-wait self-test (pa_selftest_wait_timeout):
    afterwards the error word holds PA_DEVERR_TIMEOUT."""
    check(_lib.lib().pa_selftest_wait_timeout(int(wait_ms), _stream(stream)), "pa_selftest_wait_timeout")


def get_device_error(stream=None) -> int:
    """Read and clear the device error word (synchronises the stream)."""
    code = C.c_int32(0)
    st = _lib.lib().pa_get_device_error(C.byref(code), _stream(stream))
    if st not in (_lib.PA_OK, _lib.PA_ERR_DEVICE_CHECK):
        check(st, "pa_get_device_error")
    return int(code.value)


def default_scale(head_dim: int) -> float:
    return 1.0 / math.sqrt(head_dim)
