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

def _device_of(**tensors) -> torch.device:
    """The one CUDA device that all given tensors are on."""
    device = None
    for name, t in tensors.items():
        if t is None:
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name}: expected a tensor, got {type(t).__name__}")
        if not t.is_cuda:
            raise ValueError(f"{name}: must be a CUDA tensor")
        if device is None:
            device = t.device
        elif t.device != device:
            raise ValueError(f"{name}: on {t.device}, the other tensors on {device}")
    return device


@contextlib.contextmanager
def _switched(device: torch.device, stream):
    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(int(stream), device=device)
            if stream.device != device:
                raise ValueError(f"stream on {stream.device}, the tensors on {device}")
            with torch.cuda.stream(stream):
                yield


def _on(device: torch.device, stream):
    """Makes ``device`` and ``stream`` current, so that launches and allocations belong to them."""
    if stream is None and torch.cuda.current_device() == device.index:
        return contextlib.nullcontext()
    return _switched(device, stream)


def _heads_arg(t: torch.Tensor, name: str, dtype, shape=None) -> svdq_heads:
    if t.dim() != 3:
        raise ValueError(f"{name}: expected (tokens, heads, head_dim), got shape {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.dtype not in _DTYPES:
        raise TypeError(f"{name}: must be bf16 or fp16, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.numel() == 0:
        return svdq_heads()
    if t.shape[2] > 1 and t.stride(2) != 1:
        raise ValueError(f"{name}: head_dim must be contiguous")
    st, sh = (t.stride(0) if t.shape[0] > 1 else 0), (t.stride(1) if t.shape[1] > 1 else 0)
    if st % 8 or sh % 8 or t.data_ptr() % 16:
        raise ValueError(f"{name}: needs 16-byte alignment and token and head strides that are multiples of 8 elements")
    return svdq_heads(t.data_ptr(), st, sh)


def _distinct(t: torch.Tensor, name: str) -> None:
    """Refuses an output whose elements share memory (expanded or overlapping views)."""
    extent = 1
    for stride, size in sorted((t.stride(i), t.shape[i]) for i in range(t.dim()) if t.shape[i] > 1):
        if stride < extent:
            raise ValueError(f"{name}: its elements overlap in memory")
        extent = stride * (size - 1) + extent


def _vector(t: torch.Tensor, name: str, dtype, n: int) -> int:
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if tuple(t.shape) != (n,):
        raise ValueError(f"{name}: expected shape {(n,)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t.data_ptr()


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
    device = _device_of(q=q, k=k, q_weight=q_weight, k_weight=k_weight, positions=positions, inv_freq=inv_freq,
                        pair_axis=pair_axis)
    d = svdq_qk_norm_rope_desc(q=_heads_arg(q, "q", None), eps=eps, axes=1, interleaved=interleaved, hadamard=hadamard)
    tokens, d.q_heads, dim = q.shape
    d.tokens, d.head_dim, d.dtype = tokens, dim, _DTYPES[q.dtype]
    if k is not None:
        d.k = _heads_arg(k, "k", q.dtype, (tokens, k.shape[1] if k.dim() == 3 else -1, dim))
        d.k_heads = k.shape[1]
    elif k_weight is not None:
        raise ValueError("k_weight without k")
    if q_weight is not None:
        d.q_weight = _vector(q_weight, "q_weight", q.dtype, dim)
    if k_weight is not None:
        d.k_weight = _vector(k_weight, "k_weight", q.dtype, dim)
    if inv_freq is not None:
        if positions is None:
            raise ValueError("inv_freq without positions")
        if positions.dtype != torch.int32:
            raise TypeError(f"positions: expected torch.int32, got {positions.dtype}")
        if positions.dim() not in (1, 2) or positions.shape[0] != tokens or 0 in positions.shape[1:]:
            raise ValueError(f"positions: expected (tokens,) or (tokens, axes), got {tuple(positions.shape)}")
        if positions.dim() == 2 and positions.shape[1] > 1 and positions.stride(1) != 1:
            raise ValueError("positions: the axes of a token must be contiguous")
        d.positions, d.position_stride = positions.data_ptr(), positions.stride(0)
        d.axes = positions.shape[1] if positions.dim() == 2 else 1
        d.pairs = inv_freq.shape[0] if inv_freq.dim() == 1 else -1
        d.inv_freq = _vector(inv_freq, "inv_freq", torch.float32, d.pairs)
        if pair_axis is not None:
            d.pair_axis = _vector(pair_axis, "pair_axis", torch.uint8, d.pairs)
    elif positions is not None or pair_axis is not None:
        raise ValueError("positions or pair_axis without inv_freq")
    with _on(device, stream):
        if inplace:
            _distinct(q, "q")
            if k is not None:
                _distinct(k, "k")
            q_out, k_out = q, k
            d.q_out, d.k_out = d.q, d.k
        else:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=device)
            d.q_out = svdq_heads(q_out.data_ptr(), d.q_heads * dim, dim)
            k_out = None
            if k is not None:
                k_out = torch.empty(k.shape, dtype=q.dtype, device=device)
                d.k_out = svdq_heads(k_out.data_ptr(), d.k_heads * dim, dim)
        svdq_qk_norm_rope(d)
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


def _cache_arg(cache) -> svdq_kv4_cache:
    kc, ks, vc, vs = cache
    if kc.dim() != 4:
        raise ValueError(f"k_codes: expected (pages, heads, page_size, head_dim / 2), got {tuple(kc.shape)}")
    pages, heads, page, half = kc.shape
    for name, t, n in (("k_codes", kc, half), ("k_scales", ks, half // 8), ("v_codes", vc, half),
                       ("v_scales", vs, half // 8)):
        if t.dtype != torch.uint8 and not (t.dtype == torch.float8_e4m3fn and name.endswith("scales")):
            raise TypeError(f"{name}: must be uint8" + (" or float8_e4m3fn" if name.endswith("scales") else ""))
        if tuple(t.shape) != (pages, heads, page, n):
            raise ValueError(f"{name}: expected shape {(pages, heads, page, n)}, got {tuple(t.shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name}: must be contiguous")
    return svdq_kv4_cache(kc.data_ptr(), ks.data_ptr(), vc.data_ptr(), vs.data_ptr(), pages, heads, page, 2 * half)


def kv4_append(cache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, stream=None) -> None:
    """Quantize k, v (tokens, heads, head_dim) into the cache: token t goes to slot ``slots[t]`` = page *
    page_size + offset (int64).  Slots outside the cache (-1 for padding) are skipped; the others must differ."""
    device = _device_of(k=k, v=v, slots=slots, k_codes=cache[0], k_scales=cache[1], v_codes=cache[2], v_scales=cache[3])
    c = _cache_arg(cache)
    shape = (slots.shape[0] if slots.dim() == 1 else -1, c.heads, c.head_dim)
    ka, va = _heads_arg(k, "k", None, shape), _heads_arg(v, "v", k.dtype, shape)
    with _on(device, stream):
        svdq_kv4_append(c, ka, va, shape[0], _DTYPES[k.dtype], _vector(slots, "slots", torch.int64, shape[0]))


def kv4_read(cache, slots: torch.Tensor, dtype: torch.dtype = torch.bfloat16, stream=None):
    """The keys and values that ``slots`` (int64) hold, each (tokens, heads, head_dim) in ``dtype``; exact.  A
    slot outside the cache reads as zeros."""
    if dtype not in _DTYPES:
        raise TypeError("dtype must be bf16 or fp16")
    device = _device_of(slots=slots, k_codes=cache[0], k_scales=cache[1], v_codes=cache[2], v_scales=cache[3])
    c = _cache_arg(cache)
    n = slots.shape[0] if slots.dim() == 1 else -1
    ptr = _vector(slots, "slots", torch.int64, n)
    with _on(device, stream):
        k, v = (torch.empty((n, c.heads, c.head_dim), dtype=dtype, device=device) for _ in range(2))
        row = c.heads * c.head_dim
        svdq_kv4_read(c, svdq_heads(k.data_ptr(), row, c.head_dim), svdq_heads(v.data_ptr(), row, c.head_dim), n,
                      _DTYPES[dtype], ptr)
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
    upper bound of kv_len known to the caller, only steers how the key axis is split.

    Returns out (tokens, q_heads, head_dim), with ``return_lse`` also the log sums (tokens, q_heads) fp32.  A
    query without keys gets 0 and -inf.  Tokens of no request are left as they were (in a new output:
    unspecified).
    """
    device = _device_of(q=q, kv_len=kv_len, block_table=block_table, q_start=q_start, out=out, k_codes=cache[0],
                        k_scales=cache[1], v_codes=cache[2], v_scales=cache[3])
    c = _cache_arg(cache)
    d = svdq_kv4_attention_desc(cache=c, q=_heads_arg(q, "q", None))
    tokens, heads, dim = q.shape
    if dim != c.head_dim:
        raise ValueError(f"q: head_dim {dim}, the cache's is {c.head_dim}")
    n = kv_len.shape[0] if kv_len.dim() == 1 else -1
    d.kv_len = _vector(kv_len, "kv_len", torch.int32, n)
    if block_table.dtype != torch.int32:
        raise TypeError(f"block_table: expected torch.int32, got {block_table.dtype}")
    if block_table.dim() != 2 or block_table.shape[0] != n:
        raise ValueError(f"block_table: expected ({n}, max_pages), got {tuple(block_table.shape)}")
    if block_table.shape[1] > 1 and block_table.stride(1) != 1:
        raise ValueError("block_table: a request's row must be contiguous")
    if q_start is not None:
        d.q_start = _vector(q_start, "q_start", torch.int32, n + 1)
    d.tokens, d.requests, d.q_heads, d.dtype = tokens, n, heads, _DTYPES[q.dtype]
    d.block_table, d.table_stride, d.max_pages = block_table.data_ptr(), block_table.stride(0), block_table.shape[1]
    d.max_kv_len, d.causal = int(max_kv_len or 0), causal
    d.softmax_scale = 1.0 / math.sqrt(dim) if softmax_scale is None else softmax_scale
    with _on(device, stream):
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=device)
        else:
            _distinct(out, "out")
        d.out = _heads_arg(out, "out", q.dtype, q.shape)
        lse = None
        if return_lse:
            lse = torch.empty((tokens, heads), dtype=torch.float32, device=device)
            d.lse = lse.data_ptr()
        size = svdq_kv4_attention_workspace_bytes(d)
        # From the caching allocator, on the stream in use: calls on other streams and captured graphs have their own.
        work = torch.empty(size, dtype=torch.uint8, device=device) if size else None
        svdq_kv4_attention(d, work.data_ptr() if size else None, size)
    return (out, lse) if return_lse else out
