"""The operators that follow the attention projections (include/svdq_attn.h): head norms with
rotary positions, the paged 4-bit key/value cache, and attention over it.

    q, k = qk_norm_rope(q, k, q_norm, k_norm, positions=pos, inv_freq=f, hadamard=True)
    cache = kv4_cache(pages, 64, kv_heads, 128)
    kv4_append(cache, k, v, slots)
    out = kv4_attention(q, cache, kv_len, block_table)

Tensors of heads are (tokens, heads, head_dim), bf16 or fp16, with head_dim contiguous; slices of a
packed projection output are passed as they lie.  Everything runs on the tensors' device, on
``stream`` or that device's current stream; a ``stream`` stands for ``with torch.cuda.stream(stream)``, so waits
between streams, and keeping tensors alive until a stream is done with them, are left to the caller.

Forward only, like the rest of the package: results of inputs that require grad are part of their graph, and a
backward pass through them raises; in place, or with an ``out``, such inputs are refused outside torch.no_grad().
What is written over (the cache, ``out``, heads in place) changes its version, as in torch's own in-place operations.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
from typing import NamedTuple, Optional, Sequence

import torch

import bit_quantized_linear_svdq_b200 as _base


# ----------------------------------------------------------------- 1:1 C ABI

class svdq_heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_longlong), ("head_stride", ctypes.c_longlong)]


class svdq_qk_norm_rope_desc(ctypes.Structure):
    _fields_ = [
        ("tokens", ctypes.c_int), ("q_heads", ctypes.c_int), ("k_heads", ctypes.c_int),
        ("head_dim", ctypes.c_int), ("dtype", ctypes.c_int),
        ("q", svdq_heads), ("k", svdq_heads), ("q_out", svdq_heads), ("k_out", svdq_heads),
        ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("eps", ctypes.c_float),
        ("positions", ctypes.c_void_p), ("position_stride", ctypes.c_longlong), ("axes", ctypes.c_int),
        ("inv_freq", ctypes.c_void_p), ("pair_axis", ctypes.c_void_p),
        ("pairs", ctypes.c_int), ("interleaved", ctypes.c_int), ("hadamard", ctypes.c_int),
    ]


class svdq_kv4_cache(ctypes.Structure):
    _fields_ = [
        ("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
        ("v_codes", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
        ("pages", ctypes.c_longlong), ("heads", ctypes.c_int), ("page_size", ctypes.c_int), ("head_dim", ctypes.c_int),
    ]


class svdq_kv4_attention_desc(ctypes.Structure):
    _fields_ = [
        ("cache", svdq_kv4_cache),
        ("tokens", ctypes.c_int), ("requests", ctypes.c_int), ("q_heads", ctypes.c_int), ("dtype", ctypes.c_int),
        ("q", svdq_heads), ("out", svdq_heads), ("lse", ctypes.c_void_p),
        ("kv_len", ctypes.c_void_p), ("q_start", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
        ("table_stride", ctypes.c_longlong), ("max_pages", ctypes.c_int), ("max_kv_len", ctypes.c_int),
        ("causal", ctypes.c_int), ("softmax_scale", ctypes.c_float),
    ]


def svdq_qk_norm_rope(desc: svdq_qk_norm_rope_desc, stream=None) -> None:
    _base._check(_base.load_library().svdq_qk_norm_rope(ctypes.addressof(desc), _base._stream(stream)),
                 "svdq_qk_norm_rope")


def svdq_kv4_append(cache: svdq_kv4_cache, k: svdq_heads, v: svdq_heads, tokens: int, dtype: int, slots_ptr,
                    stream=None) -> None:
    _base._check(_base.load_library().svdq_kv4_append(
        ctypes.addressof(cache), ctypes.addressof(k), ctypes.addressof(v), tokens, dtype, slots_ptr,
        _base._stream(stream)), "svdq_kv4_append")


def svdq_kv4_read(cache: svdq_kv4_cache, k_out: svdq_heads, v_out: svdq_heads, tokens: int, dtype: int, slots_ptr,
                  stream=None) -> None:
    _base._check(_base.load_library().svdq_kv4_read(
        ctypes.addressof(cache), ctypes.addressof(k_out), ctypes.addressof(v_out), tokens, dtype, slots_ptr,
        _base._stream(stream)), "svdq_kv4_read")


def svdq_kv4_attention_workspace_bytes(desc: svdq_kv4_attention_desc) -> int:
    return _base.load_library().svdq_kv4_attention_workspace_bytes(ctypes.addressof(desc))


def svdq_kv4_attention(desc: svdq_kv4_attention_desc, workspace_ptr, workspace_bytes: int, stream=None) -> None:
    _base._check(_base.load_library().svdq_kv4_attention(ctypes.addressof(desc), workspace_ptr, workspace_bytes,
                                                         _base._stream(stream)), "svdq_kv4_attention")


def svdq_kv4_attention_status() -> int:
    flags = ctypes.c_int(0)
    st = _base.load_library().svdq_kv4_attention_status(ctypes.byref(flags))
    if st not in (0, 6):
        raise _base.SvdqError(st, "svdq_kv4_attention_status")
    return flags.value


# ----------------------------------------------------------------- calls with tensors
#
# csrc/attn_torch.cpp checks the tensors, allocates outputs and workspaces on the current stream and calls the C entry
# points above: at single tokens the host's part of a call is what a user waits for.

_native = None


def _calls():
    """The extension module (raises if the library or the module has not been built)."""
    global _native
    if _native is None:
        _base.load_library()
        path = os.path.join(os.path.dirname(_base.library_path()), "_attn_torch.so")
        if not os.path.exists(path):
            raise RuntimeError(f"extension module not built: {path} is missing "
                               "(run: python -m bit_quantized_linear_svdq_b200.build)")
        loader = importlib.machinery.ExtensionFileLoader("_attn_torch", path)
        module = importlib.util.module_from_spec(importlib.util.spec_from_file_location("_attn_torch", path, loader=loader))
        loader.exec_module(module)
        _native = module
    return _native


def _run(call, name: str, where, stream, *args):
    """One call on ``stream`` (None: the current one of the device of the tensor ``where``)."""
    if stream is None:
        status, result = call(*args)
    else:
        if not isinstance(where, torch.Tensor) or not where.is_cuda:
            raise ValueError(f"{name}: expected CUDA tensors")
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device=where.device)
        if stream.device != where.device:
            raise ValueError(f"stream on {stream.device}, the tensors on {where.device}")
        with torch.cuda.stream(stream):
            status, result = call(*args)
    if status:
        raise _base.SvdqError(status, name)
    return result


# ----------------------------------------------------------------- norm, positions, rotation

def rope_frequencies(pairs: Sequence[int], theta: float = 10000.0, restart: bool = True, device="cuda"):
    """(inv_freq, pair_axis) of :func:`qk_norm_rope` for ``pairs[a]`` channel pairs on axis a: one spectrum
    per axis (``restart``), theta^(-j / pairs[a]), or one over all pairs in sections."""
    if not pairs or any(int(n) != n or n < 0 for n in pairs) or len(pairs) > 256:
        raise ValueError("pairs: one count for each axis")
    total, f, axis = sum(pairs), [], []
    for a, n in enumerate(pairs):
        start, over = (0, n) if restart else (len(f), total)
        f += [float(theta) ** (-(start + j) / over) for j in range(n)]
        axis += [a] * n
    return (torch.tensor(f, dtype=torch.float32, device=device), torch.tensor(axis, dtype=torch.uint8, device=device))


def qk_norm_rope(q: torch.Tensor, k: Optional[torch.Tensor] = None, q_weight: Optional[torch.Tensor] = None,
                 k_weight: Optional[torch.Tensor] = None, *, eps: float = 1e-6,
                 positions: Optional[torch.Tensor] = None, inv_freq: Optional[torch.Tensor] = None,
                 pair_axis: Optional[torch.Tensor] = None, interleaved: bool = False, hadamard: bool = False,
                 inplace: bool = False, stream=None):
    """RMS norm of every head (where its weight is given), rotary positions with one or several axes (where
    ``inv_freq`` is given) and the per-head Hadamard rotation (if ``hadamard``), in one pass over q and k.

    q (tokens, q_heads, head_dim), k (tokens, k_heads, head_dim) or None; weights (head_dim,); positions
    (tokens,) or (tokens, axes) int32; inv_freq (pairs,) fp32; pair_axis (pairs,) uint8, the axis of each pair
    (None: axis 0); pairs are adjacent channels if ``interleaved``, else channels p and p + pairs.  Returns
    (q, k), new and contiguous, or the arguments themselves, written over, if ``inplace`` (q and k may not overlap then).
    """
    return _run((_native or _calls()).qk_norm_rope, "svdq_qk_norm_rope", q, stream, q, k, q_weight, k_weight, eps, positions,
                inv_freq, pair_axis, interleaved, hadamard, inplace)


# ----------------------------------------------------------------- the 4-bit cache

class KV4Cache(NamedTuple):
    """The paged cache's tensors: codes (pages, heads, page_size, head_dim / 2) uint8, e4m3 scales (pages, heads,
    page_size, head_dim / 16) uint8 or float8_e4m3fn.  Any sequence of the four is taken in its place."""
    k_codes: torch.Tensor
    k_scales: torch.Tensor
    v_codes: torch.Tensor
    v_scales: torch.Tensor


def kv4_cache(pages: int, page_size: int, heads: int, head_dim: int, device="cuda") -> KV4Cache:
    """A zeroed cache of ``pages`` pages of ``page_size`` tokens."""
    if head_dim not in (64, 128):
        raise ValueError("head_dim must be 64 or 128")
    if page_size not in (16, 32, 64, 128, 256):
        raise ValueError("page_size must be 16, 32, 64, 128 or 256")
    if pages < 1 or heads < 1:
        raise ValueError("pages and heads must be at least 1")
    return KV4Cache(*(torch.zeros((pages, heads, page_size, n), dtype=torch.uint8, device=device)
                      for n in (head_dim // 2, head_dim // 16, head_dim // 2, head_dim // 16)))


def kv4_append(cache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, stream=None) -> None:
    """Quantize k, v (tokens, heads, head_dim) into the cache: token t goes to slot ``slots[t]`` = page *
    page_size + offset (int64).  Slots outside the cache (-1 for padding) are skipped; the others must differ.  The
    cache's four tensors, k, v and slots may share a buffer, but not memory.  Blocks of 16 values keep magnitudes
    from about 0.1 to 2688 (include/svdq_attn.h says what happens outside)."""
    _run((_native or _calls()).kv4_append, "svdq_kv4_append", k, stream, cache, k, v, slots)


def kv4_read(cache, slots: torch.Tensor, dtype: torch.dtype = torch.bfloat16, stream=None):
    """The keys and values that ``slots`` (int64) hold, each (tokens, heads, head_dim) in ``dtype``; exact.  A
    slot outside the cache reads as zeros."""
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        raise TypeError("dtype must be bf16 or fp16")
    return _run((_native or _calls()).kv4_read, "svdq_kv4_read", slots, stream, cache, slots, dtype is torch.float16)


def kv4_attention(q: torch.Tensor, cache, kv_len: torch.Tensor, block_table: torch.Tensor, *,
                  q_start: Optional[torch.Tensor] = None, causal: bool = True, softmax_scale: Optional[float] = None,
                  max_kv_len: Optional[int] = None, out: Optional[torch.Tensor] = None, return_lse: bool = False,
                  stream=None):
    """Attention of the new tokens q (tokens, q_heads, head_dim) over the cache.

    Request b has kv_len[b] keys (int32, the new tokens' own among them), key j in page block_table[b, j //
    page_size] (int32, (requests, max_pages)); its queries are tokens q_start[b] .. q_start[b + 1] (int32,
    (requests + 1,), ascending; None: the same number each) and stand at its last positions.  causal: a query
    sees keys up to its own position, else all.  softmax_scale defaults to 1 / sqrt(head_dim).  max_kv_len, an
    upper bound of kv_len known to the caller, only steers how the work is split.  out may not overlap any argument.

    Returns out (tokens, q_heads, head_dim), with ``return_lse`` also the log sums (tokens, q_heads) fp32.  A
    query without keys gets 0 and -inf.  Tokens of no request are left as they were (in a new output:
    unspecified).
    """
    return _run((_native or _calls()).kv4_attention, "svdq_kv4_attention", q, stream, q, cache, kv_len, block_table, q_start,
                causal, softmax_scale, max_kv_len, out, return_lse)
