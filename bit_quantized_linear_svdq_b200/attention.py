"""The operators that follow the attention projections (include/svdq_attn.h): head norms with
rotary positions, the paged 4-bit key/value cache, and attention over it.

    q, k = qk_norm_rope(q, k, q_norm, k_norm, positions=pos, inv_freq=f, hadamard=True)
    cache = kv4_cache(pages, 64, kv_heads, 128)
    kv4_append(cache, k, v, slots)
    out = kv4_attention(q, cache, kv_len, block_table)

Tensors of heads are (tokens, heads, head_dim), bf16 or fp16, with head_dim contiguous; slices of a
packed projection output are passed as they lie.  Everything runs on the tensors' device, on
``stream`` or that device's current stream.  Forward only, like the rest of the package.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import struct
from typing import NamedTuple, Optional, Sequence

import torch

import bit_quantized_linear_svdq_b200 as _base

_DTYPES = {torch.bfloat16: 0, torch.float16: 1}


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


# ----------------------------------------------------------------- argument checks
#
# At single tokens the host's part of a call is what a user waits for, so the checks below take a short path where
# everything is as it should be and look for what is wrong only where it is not; descriptions are packed as bytes.

_ROPE = struct.Struct("5iPqqPqqPqqPqqPPfPqiPP3i0P")               # svdq_qk_norm_rope_desc
_HEADS = struct.Struct("Pqq")                                     # svdq_heads
_CACHE = struct.Struct("4Pq3i0P")                                 # svdq_kv4_cache
_ATTENTION = struct.Struct("4Pq3i4x4iPqqPqqPPPPq3if")             # svdq_kv4_attention_desc

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_nothing = contextlib.nullcontext()


def _device_of(first: str, t) -> int:
    """Index of the CUDA device of a call's first tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{first}: expected a tensor, got {type(t).__name__}")
    if not t.is_cuda:
        raise ValueError(f"{first}: must be a CUDA tensor")
    return t.get_device()


def _elsewhere(name: str, t, device: int):
    """Raises for an argument that is no tensor on the call's device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a tensor, got {type(t).__name__}")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if t.get_device() != device:
        raise ValueError(f"{name}: on {t.device}, the other tensors on cuda:{device}")


@contextlib.contextmanager
def _switched(device: int, stream):
    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(int(stream), device=device)
            if stream.device.index != device:
                raise ValueError(f"stream on {stream.device}, the tensors on cuda:{device}")
            with torch.cuda.stream(stream):
                yield


def _on(device: int, stream):
    """Makes ``device`` and ``stream`` current, so that launches and allocations belong to them."""
    if stream is None and torch.cuda.current_device() == device:
        return _nothing
    return _switched(device, stream)


def _current(device: int) -> int:
    return _raw_stream(device) if _raw_stream else torch.cuda.current_stream(device).cuda_stream


def _heads_arg(t: torch.Tensor, name: str, dtype, device: int, shape=None):
    """(address, token stride, head stride) of a tensor of heads."""
    if not isinstance(t, torch.Tensor) or t.get_device() != device:
        _elsewhere(name, t, device)
    if t.dim() != 3:
        raise ValueError(f"{name}: expected (tokens, heads, head_dim), got shape {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    token, head, one = t.stride()
    address = t.data_ptr()
    if one != 1 or (token | head) & 7 or address & 15:
        n_token, n_head, n_dim = t.shape
        if t.numel() == 0:
            return 0, 0, 0
        if n_dim > 1 and one != 1:
            raise ValueError(f"{name}: head_dim must be contiguous")
        token, head = (token if n_token > 1 else 0), (head if n_head > 1 else 0)
        if (token | head) & 7 or address & 15:
            raise ValueError(f"{name}: needs 16-byte alignment and token and head strides that are multiples of 8 "
                             "elements")
    return address, token, head


def _distinct(t: torch.Tensor, name: str) -> None:
    """Refuses an output whose elements share memory (expanded or overlapping views)."""
    extent = 1
    for stride, size in sorted((t.stride(i), t.shape[i]) for i in range(t.dim()) if t.shape[i] > 1):
        if stride < extent:
            raise ValueError(f"{name}: its elements overlap in memory")
        extent = stride * (size - 1) + extent


def _vector(t: torch.Tensor, name: str, dtype, n: int, device: int) -> int:
    """Address of a contiguous vector of n elements."""
    if not isinstance(t, torch.Tensor) or t.get_device() != device:
        _elsewhere(name, t, device)
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.dim() != 1 or t.shape[0] != n:
        raise ValueError(f"{name}: expected shape {(n,)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t.data_ptr()


def _length(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a tensor, got {type(t).__name__}")
    if t.dim() != 1:
        raise ValueError(f"{name}: expected a vector, got shape {tuple(t.shape)}")
    return t.shape[0]


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
    (q, k), new and contiguous, or the arguments themselves if ``inplace``.
    """
    device = _device_of("q", q)
    dtype = q.dtype
    code = _DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"q: must be bf16 or fp16, got {dtype}")
    q_in = _heads_arg(q, "q", dtype, device)
    tokens, q_heads, dim = q.shape
    k_in, k_heads = (0, 0, 0), 0
    if k is not None:
        k_in = _heads_arg(k, "k", dtype, device)
        if k.shape[0] != tokens or k.shape[2] != dim:
            raise ValueError(f"k: expected ({tokens}, heads, {dim}), got {tuple(k.shape)}")
        k_heads = k.shape[1]
    elif k_weight is not None:
        raise ValueError("k_weight without k")
    qw = 0 if q_weight is None else _vector(q_weight, "q_weight", dtype, dim, device)
    kw = 0 if k_weight is None else _vector(k_weight, "k_weight", dtype, dim, device)
    at = stride = freq = axis = pairs = 0
    axes = 1
    if inv_freq is not None:
        if positions is None:
            raise ValueError("inv_freq without positions")
        if not isinstance(positions, torch.Tensor) or positions.get_device() != device:
            _elsewhere("positions", positions, device)
        if positions.dtype is not torch.int32:
            raise TypeError(f"positions: expected torch.int32, got {positions.dtype}")
        axes = positions.shape[1] if positions.dim() == 2 else 1
        if positions.dim() not in (1, 2) or positions.shape[0] != tokens or axes == 0:
            raise ValueError(f"positions: expected (tokens,) or (tokens, axes), got {tuple(positions.shape)}")
        if axes > 1 and positions.stride(1) != 1:
            raise ValueError("positions: the axes of a token must be contiguous")
        at, stride = positions.data_ptr(), positions.stride(0)
        pairs = _length(inv_freq, "inv_freq")
        freq = _vector(inv_freq, "inv_freq", torch.float32, pairs, device)
        if pair_axis is not None:
            axis = _vector(pair_axis, "pair_axis", torch.uint8, pairs, device)
    elif positions is not None or pair_axis is not None:
        raise ValueError("positions or pair_axis without inv_freq")
    with _on(device, stream):
        if inplace:
            _distinct(q, "q")
            if k is not None:
                _distinct(k, "k")
            q_out, k_out, q_to, k_to = q, k, q_in, k_in
        else:
            q_out, k_out, k_to = torch.empty_like(q, memory_format=torch.contiguous_format), None, k_in
            q_to = q_out.data_ptr(), q_heads * dim, dim
            if k is not None:
                k_out = torch.empty_like(k, memory_format=torch.contiguous_format)
                k_to = k_out.data_ptr(), k_heads * dim, dim
        status = _base.load_library().svdq_qk_norm_rope(
            _ROPE.pack(tokens, q_heads, k_heads, dim, code, *q_in, *k_in, *q_to, *k_to, qw, kw, eps, at, stride, axes,
                       freq, axis, pairs, interleaved, hadamard), _current(device))
    if status:
        raise _base.SvdqError(status, "svdq_qk_norm_rope")
    return q_out, k_out


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


def _cache_arg(cache, device: int):
    """Fields of svdq_kv4_cache."""
    try:
        kc, ks, vc, vs = cache
    except (TypeError, ValueError):
        raise ValueError("cache: expected (k_codes, k_scales, v_codes, v_scales)") from None
    if not isinstance(kc, torch.Tensor) or kc.get_device() != device:
        _elsewhere("k_codes", kc, device)
    if kc.dim() != 4:
        raise ValueError(f"k_codes: expected (pages, heads, page_size, head_dim / 2), got {tuple(kc.shape)}")
    codes = kc.shape
    pages, heads, page, half = codes
    scales = (pages, heads, page, half // 8)
    for name, t, shape in (("k_codes", kc, codes), ("k_scales", ks, scales), ("v_codes", vc, codes),
                           ("v_scales", vs, scales)):
        if not isinstance(t, torch.Tensor) or t.get_device() != device:
            _elsewhere(name, t, device)
        if t.dtype is not torch.uint8 and not (t.dtype is torch.float8_e4m3fn and shape is scales):
            raise TypeError(f"{name}: must be uint8" + (" or float8_e4m3fn" if shape is scales else ""))
        if t.shape != shape:
            raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name}: must be contiguous")
    return kc.data_ptr(), ks.data_ptr(), vc.data_ptr(), vs.data_ptr(), pages, heads, page, 2 * half


def kv4_append(cache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, stream=None) -> None:
    """Quantize k, v (tokens, heads, head_dim) into the cache: token t goes to slot ``slots[t]`` = page *
    page_size + offset (int64).  Slots outside the cache (-1 for padding) are skipped; the others must differ."""
    device = _device_of("k", k)
    code = _DTYPES.get(k.dtype)
    if code is None:
        raise TypeError(f"k: must be bf16 or fp16, got {k.dtype}")
    c = _cache_arg(cache, device)
    tokens = _length(slots, "slots")
    shape = (tokens, c[5], c[7])
    k_in, v_in = _heads_arg(k, "k", k.dtype, device, shape), _heads_arg(v, "v", k.dtype, device, shape)
    to = _vector(slots, "slots", torch.int64, tokens, device)
    with _on(device, stream):
        status = _base.load_library().svdq_kv4_append(_CACHE.pack(*c), _HEADS.pack(*k_in), _HEADS.pack(*v_in), tokens,
                                                      code, to, _current(device))
    if status:
        raise _base.SvdqError(status, "svdq_kv4_append")


def kv4_read(cache, slots: torch.Tensor, dtype: torch.dtype = torch.bfloat16, stream=None):
    """The keys and values that ``slots`` (int64) hold, each (tokens, heads, head_dim) in ``dtype``; exact.  A
    slot outside the cache reads as zeros."""
    code = _DTYPES.get(dtype)
    if code is None:
        raise TypeError("dtype must be bf16 or fp16")
    device = _device_of("slots", slots)
    c = _cache_arg(cache, device)
    tokens, heads, dim = _length(slots, "slots"), c[5], c[7]
    at = _vector(slots, "slots", torch.int64, tokens, device)
    with _on(device, stream):
        k = slots.new_empty((tokens, heads, dim), dtype=dtype)
        v = torch.empty_like(k)
        row = heads * dim
        status = _base.load_library().svdq_kv4_read(_CACHE.pack(*c), _HEADS.pack(k.data_ptr(), row, dim),
                                                    _HEADS.pack(v.data_ptr(), row, dim), tokens, code, at,
                                                    _current(device))
    if status:
        raise _base.SvdqError(status, "svdq_kv4_read")
    return k, v


def kv4_attention(q: torch.Tensor, cache, kv_len: torch.Tensor, block_table: torch.Tensor, *,
                  q_start: Optional[torch.Tensor] = None, causal: bool = True, softmax_scale: Optional[float] = None,
                  max_kv_len: Optional[int] = None, out: Optional[torch.Tensor] = None, return_lse: bool = False,
                  stream=None):
    """Attention of the new tokens q (tokens, q_heads, head_dim) over the cache.

    Request b has kv_len[b] keys (int32, the new tokens' own among them), key j in page block_table[b, j //
    page_size] (int32, (requests, max_pages)); its queries are tokens q_start[b] .. q_start[b + 1] (int32,
    (requests + 1,), ascending; None: the same number each) and stand at its last positions.  causal: a query
    sees keys up to its own position, else all.  softmax_scale defaults to 1 / sqrt(head_dim).  max_kv_len, an
    upper bound of kv_len known to the caller, only steers how the work is split.

    Returns out (tokens, q_heads, head_dim), with ``return_lse`` also the log sums (tokens, q_heads) fp32.  A
    query without keys gets 0 and -inf.  Tokens of no request are left as they were (in a new output:
    unspecified).
    """
    device = _device_of("q", q)
    dtype = q.dtype
    code = _DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"q: must be bf16 or fp16, got {dtype}")
    c = _cache_arg(cache, device)
    q_in = _heads_arg(q, "q", dtype, device)
    tokens, heads, dim = q.shape
    if dim != c[7]:
        raise ValueError(f"q: head_dim {dim}, the cache's is {c[7]}")
    requests = _length(kv_len, "kv_len")
    lens = _vector(kv_len, "kv_len", torch.int32, requests, device)
    if not isinstance(block_table, torch.Tensor) or block_table.get_device() != device:
        _elsewhere("block_table", block_table, device)
    if block_table.dtype is not torch.int32:
        raise TypeError(f"block_table: expected torch.int32, got {block_table.dtype}")
    if block_table.dim() != 2 or block_table.shape[0] != requests:
        raise ValueError(f"block_table: expected ({requests}, max_pages), got {tuple(block_table.shape)}")
    row, one = block_table.stride()
    pages = block_table.shape[1]
    if pages > 1 and one != 1:
        raise ValueError("block_table: a request's row must be contiguous")
    start = 0 if q_start is None else _vector(q_start, "q_start", torch.int32, requests + 1, device)
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(dim)
    with _on(device, stream):
        if out is None:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
            to = out.data_ptr(), heads * dim, dim
        else:
            to = _heads_arg(out, "out", dtype, device, q.shape)
            _distinct(out, "out")
        lse = None
        if return_lse:
            lse = q.new_empty((tokens, heads), dtype=torch.float32)
        desc = _ATTENTION.pack(*c, tokens, requests, heads, code, *q_in, *to, lse.data_ptr() if return_lse else 0, lens,
                               start, block_table.data_ptr(), row, pages, max_kv_len or 0, causal, softmax_scale)
        lib = _base.load_library()
        size = lib.svdq_kv4_attention_workspace_bytes(desc)
        # From the caching allocator, on the stream in use: calls on other streams and captured graphs have their own.
        work = q.new_empty(size, dtype=torch.uint8) if size else None
        status = lib.svdq_kv4_attention(desc, work.data_ptr() if size else None, size, _current(device))
    if status:
        raise _base.SvdqError(status, "svdq_kv4_attention")
    return (out, lse) if return_lse else out
