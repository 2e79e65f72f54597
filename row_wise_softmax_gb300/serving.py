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

import contextlib
import ctypes

import torch

from . import BF16, F16, OK, SoftmaxError, lib

__all__ = ["kv_append", "attention_packed", "attention_decode"]

_CODES = {torch.bfloat16: BF16, torch.float16: F16}
_i64, _vp = ctypes.c_int64, ctypes.c_void_p


class _Heads(ctypes.Structure):
    _fields_ = [("data", _vp), ("row_stride", _i64), ("head_stride", _i64)]


class _Cache(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("n_pages", _i64), ("page_size", _i64),
                ("n_kv_heads", _i64), ("head_dim", _i64), ("k_page_stride", _i64),
                ("k_row_stride", _i64), ("k_head_stride", _i64), ("v_page_stride", _i64),
                ("v_row_stride", _i64), ("v_head_stride", _i64), ("page_table", _vp),
                ("n_seqs", _i64), ("table_width", _i64), ("table_stride", _i64)]


_declared = None


def _lib():
    """The library, with the serving entry points' argument types declared."""
    global _declared
    if _declared is None:
        L = lib()
        hp, cp, ci = ctypes.POINTER(_Heads), ctypes.POINTER(_Cache), ctypes.c_int
        cf = ctypes.c_float
        L.softmax_kv_append.argtypes = [cp, hp, hp, hp, hp, _i64, _vp, _vp, _i64, _vp, _i64, ci,
                                        ci, _vp]
        L.softmax_kv_append.restype = ci
        L.softmax_attention_decode.argtypes = [cp, hp, hp, _vp, _i64, _vp, cf, ci, _vp,
                                               ctypes.c_size_t, _vp]
        L.softmax_attention_decode.restype = ci
        L.softmax_attention_decode_workspace.argtypes = [_i64] * 5
        L.softmax_attention_decode_workspace.restype = _i64
        L.softmax_attention_packed.argtypes = [hp, hp, hp, hp, _vp, _vp, _vp, _i64, _i64, _i64,
                                               _i64, _i64, _i64, cf, ci, ci, _vp]
        L.softmax_attention_packed.restype = ci
        _declared = L
    return _declared


def _check(name, ref, **tensors):
    """The dtype code of ``ref``, after checking that every tensor lies on its
    device, shares its dtype and has contiguous head elements."""
    code = _CODES.get(ref.dtype)
    if code is None:
        raise TypeError("%s: dtype must be bfloat16 or float16, got %s" % (name, ref.dtype))
    for key, t in tensors.items():
        if not t.is_cuda or t.device != ref.device:
            raise ValueError("%s: %s must be a CUDA tensor on %s" % (name, key, ref.device))
        if t.dtype != ref.dtype:
            raise ValueError("%s: %s must have dtype %s" % (name, key, ref.dtype))
        if t.stride(-1) != 1:
            raise ValueError("%s: %s must have contiguous head elements" % (name, key))
    return code


def _index(name, key, t, shape, device):
    if t.dtype != torch.int32 or t.device != device or tuple(t.shape) != shape:
        raise ValueError("%s: %s must be an int32 tensor of shape %s on %s" %
                         (name, key, list(shape), device))
    if t.dim() and t.numel() > 1 and t.stride(-1) != 1:
        raise ValueError("%s: %s must be contiguous" % (name, key))
    return t.data_ptr()


def _heads(t):
    return _Heads(t.data_ptr(), t.stride(0), t.stride(1))


def _cache(name, k_cache, v_cache, page_table, n_seqs):
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape:
        raise ValueError("%s: k_cache and v_cache must be [pages, page_size, kv_heads, head_dim]"
                         % name)
    if page_table.dim() != 2:
        raise ValueError("%s: page_table must be [sequences, pages]" % name)
    rows = page_table.shape[0] if n_seqs is None else n_seqs
    width = page_table.shape[1]
    _index(name, "page_table", page_table, (rows, width), k_cache.device)
    p, r, h, d = k_cache.shape
    ks, vs = k_cache.stride(), v_cache.stride()
    return _Cache(k_cache.data_ptr(), v_cache.data_ptr(), p, r, h, d, ks[0], ks[1], ks[2], vs[0],
                  vs[1], vs[2], page_table.data_ptr(), rows, width,
                  page_table.stride(0) if rows > 1 else width)


@contextlib.contextmanager
def _on(device, stream):
    """The handle of ``stream`` (a torch stream, a raw handle, or None: the
    current one), with its device current and allocations made for it."""
    with torch.cuda.device(device):
        if stream is None:
            yield torch.cuda.current_stream(device).cuda_stream
        else:
            if not hasattr(stream, "cuda_stream"):
                stream = torch.cuda.ExternalStream(int(stream), device=device)
            with torch.cuda.stream(stream):
                yield stream.cuda_stream


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
    if k.dim() != 3 or k.shape != v.shape:
        raise ValueError("kv_append: k and v must be [tokens, kv_heads, head_dim]")
    n, hk, d = k.shape
    code = _check(name, k, k=k, v=v, k_cache=k_cache, v_cache=v_cache)
    device = k.device
    cache = _cache(name, k_cache, v_cache, page_table, None)
    if cache.n_kv_heads != hk or cache.head_dim != d:
        raise ValueError("kv_append: the cache's heads do not match k")
    pos = _index(name, "positions", positions, (n,), device)
    if seq_ids is not None:
        ids = _index(name, "seq_ids", seq_ids, (n,), device)
    else:
        ids = None
        if cache.n_seqs < n:
            raise ValueError("kv_append: page_table has fewer rows than there are tokens")
    rot, freq = 0, None
    if inv_freq is not None:
        if inv_freq.dtype != torch.float64 or inv_freq.device != device or inv_freq.dim() != 1 \
                or not inv_freq.is_contiguous():
            raise ValueError("kv_append: inv_freq must be a float64 vector on %s" % device)
        rot, freq = 2 * inv_freq.numel(), inv_freq.data_ptr()
    if q is None:
        if q_out is not None:
            raise ValueError("kv_append: q_out without q")
    elif q.dim() != 3 or q.shape[0] != n or q.shape[2] != d:
        raise ValueError("kv_append: q must be [tokens, heads, head_dim]")
    else:
        _check(name, k, q=q)
        if q_out is not None:
            _check(name, k, q_out=q_out)
            if q_out.shape != q.shape:
                raise ValueError("kv_append: q_out must match q")
    with _on(device, stream) as handle:
        if q is None:
            qs = qo = None
            h = 0
        else:
            if q_out is None:
                q_out = torch.empty(q.shape, dtype=q.dtype, device=device)
            qs, qo, h = _heads(q), _heads(q_out), q.shape[1]
        st = _lib().softmax_kv_append(cache, _heads(k), _heads(v), qs, qo, h, pos, ids, n, freq,
                                     rot, 1 if interleaved else 0, code, handle)
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
    if q.dim() != 3:
        raise ValueError("attention_decode: q must be [sequences, heads, head_dim]")
    b, h, d = q.shape
    code = _check(name, q, q=q, k_cache=k_cache, v_cache=v_cache)
    device = q.device
    cache = _cache(name, k_cache, v_cache, page_table, b)
    hk = cache.n_kv_heads
    if cache.head_dim != d or hk == 0 or h == 0 or h % hk:
        raise ValueError("attention_decode: the cache's heads do not match q")
    lens = _index(name, "lengths", lengths, (b,), device)
    if out is not None:
        _check(name, q, out=out)
        if out.shape != q.shape:
            raise ValueError("attention_decode: out must match q")
    with _on(device, stream) as handle:
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=device)
        lse = torch.empty((b, h), dtype=torch.float32, device=device) if return_lse else None
        L = _lib()
        need = L.softmax_attention_decode_workspace(b, h, hk, d,
                                                    cache.table_width * cache.page_size)
        ws = torch.empty(need, dtype=torch.uint8, device=device) if need > 0 else None
        st = L.softmax_attention_decode(cache, _heads(q), _heads(out),
                                        lse.data_ptr() if return_lse else None, h, lens,
                                        d ** -0.5 if scale is None else scale, code,
                                        ws.data_ptr() if need > 0 else None, max(need, 0), handle)
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
    if q.dim() != 3 or k.dim() != 3 or k.shape != v.shape or q.shape[2] != k.shape[2]:
        raise ValueError("attention_packed: q must be [total_q, heads, head_dim], k and v "
                         "[total_k, kv_heads, head_dim]")
    n, h, d = q.shape
    m, hk = k.shape[0], k.shape[1]
    if h == 0 or hk == 0 or h % hk:
        raise ValueError("attention_packed: heads must be a multiple of kv_heads")
    code = _check(name, q, q=q, k=k, v=v)
    device = q.device
    if cu_q.dim() != 1 or cu_q.numel() < 1:
        raise ValueError("attention_packed: cu_q must be a vector of sequences + 1 bounds")
    seqs = cu_q.numel() - 1
    cq = _index(name, "cu_q", cu_q, (seqs + 1,), device)
    ck = cq if cu_k is None else _index(name, "cu_k", cu_k, (seqs + 1,), device)
    if out is not None:
        _check(name, q, out=out)
        if out.shape != q.shape:
            raise ValueError("attention_packed: out must match q")
    with _on(device, stream) as handle:
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=device)
        lse = torch.empty((n, h), dtype=torch.float32, device=device) if return_lse else None
        st = _lib().softmax_attention_packed(_heads(q), _heads(k), _heads(v), _heads(out),
                                            lse.data_ptr() if return_lse else None, cq, ck, seqs,
                                            n, m, h, hk, d, d ** -0.5 if scale is None else scale,
                                            1 if causal else 0, code, handle)
    if st != OK:
        raise SoftmaxError(st, name)
    return (out, lse) if return_lse else out
