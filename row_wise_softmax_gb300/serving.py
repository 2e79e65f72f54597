"""Serving operators: paged key/value cache and packed prompts, grouped heads.

    kv_append(k, v, k_cache, v_cache, page_table, positions, ...)   rotate and append
    attention_packed(q, k, v, cu_q, cu_k, ...)                      whole prompts
    attention_decode(q, k_cache, v_cache, page_table, lengths, ...) one new token each

Argument checks and marshalling only, as in the rest of the package; the
operators are declared in include/softmax.h.  Every tensor lives on one CUDA
device; the work is queued on ``stream`` (default: torch's current stream of
that device) without synchronising, and outputs that a call allocates are
allocated for that stream.
"""
from __future__ import annotations

import ctypes
import functools
import struct

import torch

from . import BF16, F16, OK, SoftmaxError, lib

__all__ = ["kv_append", "attention_packed", "attention_decode"]

_CODES = {torch.bfloat16: BF16, torch.float16: F16}

# softmax_heads_t and softmax_paged_cache_t, packed: the calls of one decoding
# step are short, and building ctypes structures costs more than they do.
_HEADS = struct.Struct("=Qqq").pack
_CACHE = struct.Struct("=QQ10qQ3q").pack

_declared = None


def _lib():
    """The library, with the serving entry points' argument types declared."""
    global _declared
    if _declared is None:
        L = lib()
        i64, vp, ci, cf, sp = (ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_float,
                               ctypes.c_char_p)            # sp: a packed structure
        L.softmax_kv_append.argtypes = [sp, sp, sp, sp, sp, i64, vp, vp, i64, vp, i64, ci, ci, vp]
        L.softmax_kv_append.restype = ci
        L.softmax_attention_decode.argtypes = [sp, sp, sp, vp, i64, vp, cf, ci, vp,
                                               ctypes.c_size_t, vp]
        L.softmax_attention_decode.restype = ci
        L.softmax_attention_decode_workspace.argtypes = [i64] * 5
        L.softmax_attention_decode_workspace.restype = i64
        L.softmax_attention_packed.argtypes = [sp, sp, sp, sp, vp, vp, vp, i64, i64, i64, i64, i64,
                                               i64, cf, ci, ci, vp, ctypes.c_size_t, vp]
        L.softmax_attention_packed.restype = ci
        L.softmax_attention_packed_workspace.argtypes = [i64] * 6
        L.softmax_attention_packed_workspace.restype = i64
        _declared = L
    return _declared


def _refuse(name, key, t, dtype, device):
    """What is wrong with a [rows, heads, head_dim] tensor (or a cache)."""
    if t.get_device() != device:
        return ValueError("%s: %s must be a tensor on cuda:%d" % (name, key, device))
    if t.dtype is not dtype:
        return ValueError("%s: %s must have dtype %s" % (name, key, dtype))
    return ValueError("%s: %s must have contiguous head elements" % (name, key))


def _heads(name, key, t, dtype, device):
    """softmax_heads_t of a [rows, heads, head_dim] tensor."""
    row, head, one = t.stride()
    if one != 1 or t.dtype is not dtype or t.get_device() != device:
        raise _refuse(name, key, t, dtype, device)
    return _HEADS(t.data_ptr(), row, head)


def _index(name, key, t, n, device):
    """The address of an int32 vector of n elements."""
    if t.dtype is not torch.int32 or t.get_device() != device or t.shape != (n,) or \
            (n > 1 and t.stride(0) != 1):
        raise ValueError("%s: %s must be a contiguous int32 tensor of shape [%d] on cuda:%d" %
                         (name, key, n, device))
    return t.data_ptr()


def _cache(name, k, v, table, shape, dtype, device):
    """softmax_paged_cache_t of two caches (``shape``: k's) and a page table."""
    if len(shape) != 4 or v.shape != shape:
        raise ValueError("%s: k_cache and v_cache must be [pages, page_size, kv_heads, head_dim]"
                         % name)
    if table.dtype is not torch.int32 or table.get_device() != device or table.dim() != 2:
        raise ValueError("%s: page_table must be an int32 tensor [sequences, pages] on cuda:%d" %
                         (name, device))
    kp, kr, kh, k1 = k.stride()
    vp, vr, vh, v1 = v.stride()
    if k1 != 1 or k.dtype is not dtype or k.get_device() != device:
        raise _refuse(name, "k_cache", k, dtype, device)
    if v1 != 1 or v.dtype is not dtype or v.get_device() != device:
        raise _refuse(name, "v_cache", v, dtype, device)
    rows, width = table.shape
    step, one = table.stride()
    if width > 1 and one != 1:
        raise ValueError("%s: page_table's rows must be contiguous" % name)
    return _CACHE(k.data_ptr(), v.data_ptr(), *shape, kp, kr, kh, vp, vr, vh, table.data_ptr(),
                  rows, width, step if rows > 1 else width)


_current = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream

# A contiguous tensor on the current device.  torch's allocation without its
# dispatcher, where torch offers that: between two kernel launches
# torch.empty_like costs 4.7 us of host time, this 1.4 (attention_decode of 8
# sequences: 13.1 us of host time a call, then 10.4).
try:
    from torch._C._dynamo.guards import _empty_strided_cuda
except ImportError:
    def _empty_strided_cuda(size, stride, dtype):
        return torch.empty_strided(size, stride, dtype=dtype, device="cuda")


def _empty3(shape, dtype):
    a, b, c = shape
    return _empty_strided_cuda((a, b, c), (b * c, c, 1), dtype)


def _elsewhere(name, device, stream, call):
    """call() with CUDA device ``device`` and ``stream`` (a torch stream, a raw
    handle, or None: the device's current one) current, so that what it
    allocates is allocated for that stream."""
    if device < 0:
        raise ValueError("%s: expects CUDA tensors" % name)
    with torch.cuda.device(device):
        if stream is None:
            return call()
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=device)
        with torch.cuda.stream(stream):
            return call()


def _code(name, dtype):
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError("%s: dtype must be bfloat16 or float16, got %s" % (name, dtype))
    return code


@functools.lru_cache(maxsize=256)
def _decode_workspace(device, b, h, hk, d, capacity):
    """Workspace bytes of a decode call of these sizes (``device``: current)."""
    return _lib().softmax_attention_decode_workspace(b, h, hk, d, capacity)


@functools.lru_cache(maxsize=256)
def _packed_workspace(device, seqs, n, m, h, hk, d):
    """Workspace bytes of a packed call of these sizes (``device``: current)."""
    return _lib().softmax_attention_packed_workspace(seqs, n, m, h, hk, d)


def kv_append(k, v, k_cache, v_cache, page_table, positions, seq_ids=None, q=None, q_out=None,
              inv_freq=None, interleaved: bool = False, stream=None):
    """Rotate new tokens' keys (and queries) by their positions, and put keys
    and values into the paged cache.

    k, v       [tokens, kv_heads, head_dim]; q, q_out [tokens, heads, head_dim]
    caches     [pages, page_size, kv_heads, head_dim], any strides of the
               first three dimensions
    page_table int32 [sequences, pages of a sequence]
    positions  int32 [tokens]; negative: padding, nothing is written
    seq_ids    int32 [tokens], each token's row of page_table (None: token t
               belongs to sequence t)
    inv_freq   float64 [rot_dim / 2], radians per position (None: no rotation);
               pairs (i, i + rot_dim / 2), or (2i, 2i + 1) when interleaved

    Returns the rotated queries (``q_out``, which may be q itself, or a new
    tensor), or None without q.
    """
    name = "kv_append"
    device = k.get_device()
    if stream is not None or device < 0 or device != _current():
        return _elsewhere(name, device, stream, lambda: kv_append(
            k, v, k_cache, v_cache, page_table, positions, seq_ids, q, q_out, inv_freq,
            interleaved))
    shape = k.shape
    if len(shape) != 3 or v.shape != shape:
        raise ValueError("kv_append: k and v must be [tokens, kv_heads, head_dim]")
    n, hk, d = shape
    dtype = k.dtype
    code = _CODES.get(dtype) or _code(name, dtype)
    shape = k_cache.shape
    cache = _cache(name, k_cache, v_cache, page_table, shape, dtype, device)
    if shape[2] != hk or shape[3] != d:
        raise ValueError("kv_append: the cache's heads do not match k")
    pos = _index(name, "positions", positions, n, device)
    ids = None
    if seq_ids is not None:
        ids = _index(name, "seq_ids", seq_ids, n, device)
    elif page_table.shape[0] < n:
        raise ValueError("kv_append: page_table has fewer rows than there are tokens")
    rot, freq = 0, None
    if inv_freq is not None:
        if inv_freq.dtype is not torch.float64 or inv_freq.get_device() != device or \
                inv_freq.dim() != 1 or not inv_freq.is_contiguous():
            raise ValueError("kv_append: inv_freq must be a float64 vector on cuda:%d" % device)
        rot, freq = 2 * inv_freq.shape[0], inv_freq.data_ptr()
    h, qs, qo = 0, None, None
    if q is not None:
        shape = q.shape
        if len(shape) != 3 or shape[0] != n or shape[2] != d:
            raise ValueError("kv_append: q must be [tokens, heads, head_dim]")
        h = shape[1]
        if q_out is None:
            q_out = _empty3(shape, dtype)
        elif q_out.shape != shape:
            raise ValueError("kv_append: q_out must match q")
        qs = _heads(name, "q", q, dtype, device)
        qo = _heads(name, "q_out", q_out, dtype, device)
    elif q_out is not None:
        raise ValueError("kv_append: q_out without q")
    st = (_declared or _lib()).softmax_kv_append(
        cache, _heads(name, "k", k, dtype, device), _heads(name, "v", v, dtype, device), qs, qo, h,
        pos, ids, n, freq, rot, 1 if interleaved else 0, code, _raw_stream(device))
    if st != OK:
        raise SoftmaxError(st, name)
    return q_out


def attention_decode(q, k_cache, v_cache, page_table, lengths, scale: float | None = None,
                     out=None, return_lse: bool = False, stream=None):
    """softmax(scale q K^T) V of one query row per sequence over its cached
    tokens.

    q          [sequences, heads, head_dim]; ``out`` (optional) like q, may be q
    caches     [pages, page_size, kv_heads, head_dim], any strides of the
               first three dimensions; heads is a multiple of kv_heads
    page_table int32 [sequences, pages of a sequence]
    lengths    int32 [sequences]: cached tokens of each; 0 gives NaN

    scale defaults to 1 / sqrt(head_dim).  Returns out, or (out, lse) with lse
    float32 [sequences, heads].
    """
    name = "attention_decode"
    device = q.get_device()
    if stream is not None or device < 0 or device != _current():
        return _elsewhere(name, device, stream, lambda: attention_decode(
            q, k_cache, v_cache, page_table, lengths, scale, out, return_lse))
    qshape = q.shape
    if len(qshape) != 3:
        raise ValueError("attention_decode: q must be [sequences, heads, head_dim]")
    b, h, d = qshape
    dtype = q.dtype
    code = _CODES.get(dtype) or _code(name, dtype)
    shape = k_cache.shape
    cache = _cache(name, k_cache, v_cache, page_table, shape, dtype, device)
    _, size, hk, dim = shape
    if dim != d or hk == 0 or h == 0 or h % hk:
        raise ValueError("attention_decode: the cache's heads do not match q")
    rows, width = page_table.shape
    if rows != b:
        raise ValueError("attention_decode: page_table must have a row for each query")
    lens = _index(name, "lengths", lengths, b, device)
    if out is None:
        out = _empty3(qshape, dtype)
    elif out.shape != qshape:
        raise ValueError("attention_decode: out must match q")
    lse = _empty_strided_cuda((b, h), (h, 1), torch.float32) if return_lse else None
    need = _decode_workspace(device, b, h, hk, d, width * size)
    ws = _empty_strided_cuda((need,), (1,), torch.uint8) if need > 0 else None
    st = (_declared or _lib()).softmax_attention_decode(
        cache, _heads(name, "q", q, dtype, device), _heads(name, "out", out, dtype, device),
        lse.data_ptr() if return_lse else None, h, lens, d ** -0.5 if scale is None else scale,
        code, ws.data_ptr() if need > 0 else None, need if need > 0 else 0, _raw_stream(device))
    if st != OK:
        raise SoftmaxError(st, name)
    return (out, lse) if return_lse else out


def attention_packed(q, k, v, cu_q, cu_k=None, scale: float | None = None, causal: bool = True,
                     out=None, return_lse: bool = False, stream=None):
    """softmax(scale q k^T, mask) v of sequences packed one behind the other.

    q          [total_q, heads, head_dim]; k, v [total_k, kv_heads, head_dim];
               heads is a multiple of kv_heads; any strides of the first two
               dimensions
    cu_q, cu_k int32 [sequences + 1]: sequence s has rows cu[s] to cu[s + 1]
               (cu_k None: cu_q)
    causal     key j is visible to query i iff j <= i + (n_k - n_q), counted
               within the sequence (the last query sees every key)

    scale defaults to 1 / sqrt(head_dim).  A query that sees no key gives NaN;
    rows of ``out`` in no sequence are left as they were.  Returns out, or
    (out, lse) with lse float32 [total_q, heads].
    """
    name = "attention_packed"
    device = q.get_device()
    if stream is not None or device < 0 or device != _current():
        return _elsewhere(name, device, stream, lambda: attention_packed(
            q, k, v, cu_q, cu_k, scale, causal, out, return_lse))
    qshape, shape = q.shape, k.shape
    if len(qshape) != 3 or len(shape) != 3 or v.shape != shape:
        raise ValueError("attention_packed: q must be [total_q, heads, head_dim], k and v "
                         "[total_k, kv_heads, head_dim]")
    n, h, d = qshape
    m, hk, dim = shape
    if dim != d or h == 0 or hk == 0 or h % hk:
        raise ValueError("attention_packed: heads must be a multiple of kv_heads, and head_dim "
                         "the same")
    dtype = q.dtype
    code = _CODES.get(dtype) or _code(name, dtype)
    seqs = cu_q.numel() - 1
    if seqs < 0:
        raise ValueError("attention_packed: cu_q must be a vector of sequences + 1 bounds")
    cq = _index(name, "cu_q", cu_q, seqs + 1, device)
    ck = cq if cu_k is None else _index(name, "cu_k", cu_k, seqs + 1, device)
    if out is None:
        out = _empty3(qshape, dtype)
    elif out.shape != qshape:
        raise ValueError("attention_packed: out must match q")
    lse = _empty_strided_cuda((n, h), (h, 1), torch.float32) if return_lse else None
    need = _packed_workspace(device, seqs, n, m, h, hk, d)
    ws = _empty_strided_cuda((need,), (1,), torch.uint8) if need > 0 else None
    st = (_declared or _lib()).softmax_attention_packed(
        _heads(name, "q", q, dtype, device), _heads(name, "k", k, dtype, device),
        _heads(name, "v", v, dtype, device), _heads(name, "out", out, dtype, device),
        lse.data_ptr() if return_lse else None, cq, ck, seqs, n, m, h, hk, d,
        d ** -0.5 if scale is None else scale, 1 if causal else 0, code,
        ws.data_ptr() if need > 0 else None, need if need > 0 else 0, _raw_stream(device))
    if st != OK:
        raise SoftmaxError(st, name)
    return (out, lse) if return_lse else out
