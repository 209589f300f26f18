"""Torch-tensor binding of the paged-KV C ABI (argument marshalling only).

Every function passes ``data_ptr()`` values, sizes and the current CUDA
stream to the function of the same name in ``include/pa.h``; all work runs in
the library's kernels.  Tensors must be contiguous CUDA tensors of the
documented shapes; int32 index tensors live on the same device.
"""
from __future__ import annotations

import ctypes as C
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


def make_workspace(q, block_tables, block_size, split_tokens=0):
    """Allocate (with torch) the scratch that :func:`decode` needs, or None."""
    B, hq, d = q.shape
    n = decode_workspace_size(B, hq, d, int(block_tables.shape[1]), block_size, split_tokens)
    if n == 0:
        return None
    return torch.empty(n, dtype=torch.uint8, device=q.device)


def decode(q, k_cache, v_cache, block_tables, context_lens, scale, out=None, split_tokens=0, workspace=None,
           stream=None):
    if out is None:
        out = torch.empty_like(q)
    _check_decode(q, k_cache, v_cache, block_tables, context_lens, out)
    if workspace is None:
        workspace = make_workspace(q, block_tables, k_cache.shape[1], split_tokens)
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
        out = torch.empty_like(q)
    if dq != d:
        raise ValueError("head_dim mismatch")
    _check_attention(q, k_cache, v_cache, out)
    _check_index(q, "block_tables", block_tables, B, table=True)
    _check_index(q, "context_lens", context_lens, B)
    maxblk = int(block_tables.shape[1])
    if workspace is None:
        n = verify_workspace_size(B, ql, hq, d, maxblk, bs, split_tokens)
        workspace = torch.empty(n, dtype=torch.uint8, device=q.device) if n else None
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
    of ``q``, the prefix's K/V and the previous use of ``workspace``."""
    nb, bs, hkv, d = _cache_dims(k_cache)
    B, hq, dq = q.shape
    if dq != d:
        raise ValueError("head_dim mismatch")
    if out is None:
        out = torch.empty_like(q)
    _check_attention(q, k_cache, v_cache, out)
    _check_index(q, "block_tables", block_tables, B, table=True)
    _check_index(q, "context_lens", context_lens, B)
    if prefix_blocks.device != q.device or prefix_blocks.numel() < int(prefix_len) // bs:
        raise ValueError("prefix_blocks must hold prefix_len / block_size block ids on q's device")
    maxblk = int(block_tables.shape[1])
    if workspace is None:
        n = decode_shared_prefix_workspace_size(B, hq, d, maxblk, bs, int(prefix_len), split_tokens)
        workspace = torch.empty(max(n, 1), dtype=torch.uint8, device=q.device)
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
        out = torch.empty_like(q)
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
        out = torch.empty_like(q)
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


def _check_current(t: torch.Tensor):
    """The library launches on the current device: a tensor elsewhere would be another GPU's memory."""
    if t.is_cuda and t.device.index != torch.cuda.current_device():
        raise ValueError(f"tensors are on {t.device}, but the current device is cuda:{torch.cuda.current_device()}")


def rope_table(max_position: int, rot_dim: int, base: float = 10000.0, device=None) -> torch.Tensor:
    """fp32 [max_position, rot_dim], cosines then sines of ``position * base^(-2j/rot_dim)``: the table
    :func:`norm_rope_and_cache` reads.  The angles are taken in 64 bits: in 32 those of far positions lose the
    digits that matter."""
    j = torch.arange(rot_dim // 2, dtype=torch.float64, device=device)
    angle = torch.arange(max_position, dtype=torch.float64, device=device)[:, None] * base ** (-2.0 * j / rot_dim)
    return torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32)


def _token_rows(t: torch.Tensor, name: str, heads: int, d: int, dtype, device) -> int:
    """Token stride (elements) of [num_tokens, heads, head_dim] whose heads are contiguous."""
    if t.dtype != dtype:
        raise TypeError(f"{name} ({t.dtype}) must have the cache's dtype ({dtype})")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not {device}")
    row = heads * d
    if t.is_contiguous():
        stride = row
    else:
        s0, s1, s2 = t.stride()
        if s2 != 1 or (heads > 1 and s1 != d):
            raise ValueError(f"{name}: the heads of a token must be contiguous")
        stride = s0 if t.shape[0] > 1 else row
    if stride < row or stride % 8:
        raise ValueError(f"{name}: tokens must be at least a row, and a multiple of 8 elements, apart")
    return stride


_Sections = C.c_int32 * 3


def norm_rope_and_cache(q, k, v, positions, cos_sin, slot_mapping, k_cache, v_cache, q_weight=None, k_weight=None,
                        eps=1e-6, sections=None, interleaved=False, out=None, stream=None):
    """pa_norm_rope_and_cache: per-head norm (with ``q_weight``/``k_weight``) and rotary position of new queries and
    keys, keys and values into their slots; returns the queries.

    ``q``/``k``/``v`` may be views of one projection's rows.  ``positions``: int32 [num_tokens], or
    [axes, num_tokens] with ``sections`` (pairs per axis).  ``out`` may be ``q`` if that is contiguous."""
    nb, bs, hkv, d = _cache_dims(k_cache)
    _check_caches(k_cache, v_cache)
    dtype, device = k_cache.dtype, k_cache.device
    if q.dim() != 3 or q.shape[2] != d:
        raise ValueError("q is [num_tokens, q_heads, head_dim] of the cache's head_dim")
    T, hq, _ = q.shape
    if k.shape != (T, hkv, d) or v.shape != (T, hkv, d):
        raise ValueError("k and v are [num_tokens, kv_heads, head_dim] of the cache, as many tokens as q")
    qs = _token_rows(q, "q", hq, d, dtype, device)
    ks = _token_rows(k, "k", hkv, d, dtype, device)
    vs = _token_rows(v, "v", hkv, d, dtype, device)
    pshape = positions.shape
    axes = 1 if len(pshape) == 1 else pshape[0] if len(pshape) == 2 else 0
    if not 1 <= axes <= 3 or pshape[-1] != T or positions.device != device:
        raise ValueError("positions is [num_tokens] or [1 to 3 axes, num_tokens] on q's device")
    if cos_sin.dim() != 2 or cos_sin.dtype != torch.float32 or cos_sin.device != device:
        raise ValueError("cos_sin is fp32 [max_position, rot_dim] on q's device")
    max_pos, rot = cos_sin.shape
    sec = None
    if sections is None:
        if axes > 1:
            raise ValueError("several axes need their sections")
    elif len(sections) != axes or min(sections) < 0 or sum(sections) != rot // 2:
        raise ValueError(f"sections are {axes} counts of pairs, rot_dim / 2 = {rot // 2} together")
    else:
        sec = _Sections(*sections)
    for w, n in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None and (w.shape != (d,) or w.dtype != dtype or w.device != device):
            raise ValueError(f"{n} is [head_dim] of q's dtype and device")
    _check_index(k_cache, "slot_mapping", slot_mapping, T)
    if out is None:
        out = torch.empty((T, hq, d), dtype=dtype, device=device)
    elif out.shape != (T, hq, d) or out.dtype != dtype or out.device != device:
        raise ValueError("out must have q's shape, dtype and device")
    _check_current(q)
    _keep(out)
    _launch(
        "pa_norm_rope_and_cache", _dev_rows(q, "q"), _dev_rows(k, "k"), _dev_rows(v, "v"), qs, ks, vs,
        _dev(q_weight, "q_weight") if q_weight is not None else None,
        _dev(k_weight, "k_weight") if k_weight is not None else None, eps, _i32(positions, "positions"), axes, sec,
        _dev(cos_sin, "cos_sin"), max_pos, rot, 1 if interleaved else 0, _i32(slot_mapping, "slot_mapping"), T, hq,
        _dev(out, "out"), _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"), nb, bs, hkv, d, dtype_code(dtype),
        _stream(stream))
    return out


def _dev_rows(t: torch.Tensor, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.data_ptr()


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


def verify_tree(q, q_start, tree_mask, context_lens, k_cache, v_cache, block_tables, scale, max_q_len, out=None,
                split_tokens=0, workspace=None, stream=None):
    """pa_verify_tree: ``q`` is [total_q, q_heads, head_dim], packed by ``q_start``; bit m of ``tree_mask[i]`` (int64)
    lets row i see its request's node m.  Every row sees the context before the draft."""
    nb, bs, hkv, d = _cache_dims(k_cache)
    if q.dim() != 3 or q.shape[2] != d:
        raise ValueError("q is [total_q, q_heads, head_dim] of the cache's head_dim")
    T, hq, _ = q.shape
    R = int(context_lens.shape[0])
    if out is None:
        out = torch.empty_like(q)
    _check_attention(q, k_cache, v_cache, out)
    _check_index(q, "context_lens", context_lens, R)
    _check_index(q, "q_start", q_start, R + 1)
    _check_index(q, "block_tables", block_tables, R, table=True)
    _check_index(q, "tree_mask", tree_mask, T)
    if tree_mask.dtype != torch.int64:
        raise TypeError("tree_mask must be int64")
    _check_current(q)
    maxblk = int(block_tables.shape[1])
    if workspace is None:
        n = verify_tree_workspace_size(R, T, int(max_q_len), hq, hkv, d, maxblk, bs, split_tokens)
        workspace = torch.empty(n, dtype=torch.uint8, device=q.device) if n else None
    ws_ptr, ws_bytes = (workspace.data_ptr(), workspace.numel() * workspace.element_size()) \
        if workspace is not None else (None, 0)
    _keep(out, workspace)
    _launch(
        "pa_verify_tree", _dev(q, "q"), _i32(q_start, "q_start"), _dev(tree_mask, "tree_mask"),
        _i32(context_lens, "context_lens"), _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"),
        _i32(block_tables, "block_tables"), maxblk, R, T, int(max_q_len), hq, hkv, d, bs, nb, float(scale),
        int(split_tokens), ws_ptr, ws_bytes, _dev(out, "out"), dtype_code(q.dtype), _stream(stream))
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


def _check_scores(ref, scores, hkv: int, score_rows, num_seqs: int, name="scores"):
    if scores.dim() != 3 or scores.shape[1] != hkv or scores.dtype != torch.float32 or scores.device != ref.device:
        raise ValueError(f"{name} is fp32 [rows, kv_heads, length] on {ref.device}")
    if score_rows is not None:
        _check_index(ref, "score_rows", score_rows, num_seqs)
    elif scores.shape[0] < num_seqs:
        raise ValueError(f"{name} has fewer rows than there are requests")


def decode_accumulate(q, k_cache, v_cache, block_tables, context_lens, scale, scores, score_rows=None,
                      scores_out=None, out=None, split_tokens=0, workspace=None, stream=None):
    """pa_decode_accumulate: :func:`decode`, and each cached token's attention weight (summed over the query heads of
    its KV head) added to its score.  ``scores``: fp32 [rows, kv_heads, length], request r's row is ``score_rows[r]``
    (None: r; negative: no score).  ``scores_out`` None: in place.  Returns (out, scores_out)."""
    nb, bs, hkv, d = _cache_dims(k_cache)
    if out is None:
        out = torch.empty_like(q)
    _check_decode(q, k_cache, v_cache, block_tables, context_lens, out)
    B, hq, _ = q.shape
    if scores_out is None:
        scores_out = scores
    _check_scores(q, scores, hkv, score_rows, B)
    if scores_out.shape != scores.shape:
        raise ValueError("scores_out must have scores' shape")
    _check_scores(q, scores_out, hkv, score_rows, B, "scores_out")
    _check_current(q)
    maxblk = int(block_tables.shape[1])
    if workspace is None:
        n = decode_accumulate_workspace_size(B, hq, hkv, d, maxblk, bs, split_tokens)
        workspace = torch.empty(max(n, 1), dtype=torch.uint8, device=q.device)
    _keep(out, workspace)
    _launch(
        "pa_decode_accumulate", _dev(q, "q"), _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"),
        _i32(block_tables, "block_tables"), maxblk, _i32(context_lens, "context_lens"), B, hq, hkv, d, bs, nb,
        float(scale), int(split_tokens), _dev(scores, "scores"),
        _i32(score_rows, "score_rows") if score_rows is not None else None, int(scores.shape[0]),
        int(scores.shape[2]), _dev(scores_out, "scores_out"), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _dev(out, "out"), dtype_code(q.dtype), _stream(stream))
    return out, scores_out


def evict_select(scores, context_lens, sink, heavy, recent, score_rows=None, keep=None, keep_lens=None, stream=None):
    """pa_evict_select: per request and KV head the tokens a budget of ``sink + heavy + recent`` keeps, ascending:
    the first, the last, and the best scored between.  Returns (keep int32 [num_seqs, kv_heads, budget], -1 behind;
    keep_lens int32 [num_seqs])."""
    if scores.dim() != 3:
        raise ValueError("scores is fp32 [rows, kv_heads, length]")
    B, hkv = int(context_lens.shape[0]), int(scores.shape[1])
    _check_scores(scores, scores, hkv, score_rows, B)
    _check_index(scores, "context_lens", context_lens, B)
    if min(sink, heavy, recent) < 0 or sink + heavy + recent < 1:
        raise ValueError("sink, heavy and recent are counts, at least one token together")
    budget = int(sink) + int(heavy) + int(recent)
    if keep is None:
        keep = torch.empty((B, hkv, budget), dtype=torch.int32, device=scores.device)
    elif keep.shape != (B, hkv, budget) or keep.device != scores.device:
        raise ValueError(f"keep is [{B}, {hkv}, {budget}] on {scores.device}")
    if keep_lens is None:
        keep_lens = torch.empty(B, dtype=torch.int32, device=scores.device)
    _check_index(scores, "keep_lens", keep_lens, B)
    _check_current(scores)
    _keep(keep, keep_lens)
    _launch(
        "pa_evict_select", _dev(scores, "scores"), _i32(score_rows, "score_rows") if score_rows is not None else None,
        int(scores.shape[0]), hkv, int(scores.shape[2]), _i32(context_lens, "context_lens"), B, int(sink), int(heavy),
        int(recent), _i32(keep, "keep"), _i32(keep_lens, "keep_lens"), _stream(stream))
    return keep, keep_lens


def compact_kv(k_cache, v_cache, block_tables, context_lens, keep, keep_lens, base=None, scores=None, score_rows=None,
               stream=None):
    """pa_compact_kv: token ``base[r] + i`` of each sequence becomes its token ``base[r] + keep[r, g, i]``, in place
    (``keep``: int32 [num_seqs, 1 or kv_heads, max_keep], ``i <= keep[i]``); with ``scores``, those too, and zeros
    behind them."""
    nb, bs, hkv, d = _cache_dims(k_cache)
    _check_caches(k_cache, v_cache)
    B = int(context_lens.shape[0])
    _check_index(k_cache, "block_tables", block_tables, B, table=True)
    _check_index(k_cache, "context_lens", context_lens, B)
    if keep.dim() != 3 or keep.shape[0] != B or keep.shape[1] not in (1, hkv) or keep.device != k_cache.device:
        raise ValueError("keep is int32 [num_seqs, 1 or kv_heads, max_keep] on the cache's device")
    _check_index(k_cache, "keep_lens", keep_lens, B)
    if base is not None:
        _check_index(k_cache, "base", base, B)
    if scores is not None:
        _check_scores(k_cache, scores, hkv, score_rows, B)
    _check_current(k_cache)
    if keep.shape[2] == 0:
        if scores is not None:
            raise ValueError("keep has no entries")
        return
    with_rows = scores is not None and score_rows is not None
    _launch(
        "pa_compact_kv", _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"), _i32(block_tables, "block_tables"),
        int(block_tables.shape[1]), _i32(context_lens, "context_lens"), _i32(keep, "keep"), int(keep.shape[1]),
        int(keep.shape[2]), _i32(keep_lens, "keep_lens"), _i32(base, "base") if base is not None else None, B, nb, bs,
        hkv, d, dtype_code(k_cache.dtype), _dev(scores, "scores") if scores is not None else None,
        _i32(score_rows, "score_rows") if with_rows else None, int(scores.shape[0]) if scores is not None else 0,
        int(scores.shape[2]) if scores is not None else 0, _stream(stream))


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
