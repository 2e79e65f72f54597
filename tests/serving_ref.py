"""Plain float64 forms of the serving operators, for the tests.

Test infrastructure only: numpy on the CPU, loops over sequences, no code
shared with the kernels.  16-bit tensors come in as float64 arrays of their
exact values.
"""
import numpy as np

from oracle import attention as oatt


def rotate(x, positions, inv_freq, interleaved):
    """x [tokens, heads, dim] with its first 2 len(inv_freq) elements turned
    by positions * inv_freq (angles reduced with integers: position and
    frequency as exact fractions of a turn are not needed at 64 bits for
    positions below 2^31 and the tolerances of the tests)."""
    half = len(inv_freq)
    ang = np.asarray(positions, np.float64)[:, None, None] * np.asarray(inv_freq, np.float64)
    c, s = np.cos(ang), np.sin(ang)
    y = np.array(x, np.float64)
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a * c - b * s, a * s + b * c
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y[..., :half], y[..., half:2 * half] = a * c - b * s, a * s + b * c
    return y


def attend(q, k, v, scale, offset=None):
    """One sequence: q [n_q, H, d], k and v [n_k, Hk, d] -> (o, lse, mag) with
    mag the same weights applied to |v|; offset None: every key visible."""
    n_q, h, d = q.shape
    g = h // k.shape[1]
    qh = q.transpose(1, 0, 2)
    kh, vh = (np.repeat(a.transpose(1, 0, 2), g, 0) for a in (k, v))
    causal, off = offset is not None, offset or 0
    o = oatt.attention(qh, kh, vh, scale, causal, off)
    mag = oatt.attention(qh, kh, np.abs(vh), scale, causal, off)
    lse = oatt.logsumexp(qh, kh, scale, causal, off)
    return o.transpose(1, 0, 2), lse.T, mag.transpose(1, 0, 2)


def packed(q, k, v, cu_q, cu_k, scale, causal):
    o, mag = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    lse = np.full(q.shape[:2], np.nan)
    for a, b, c, e in zip(cu_q[:-1], cu_q[1:], cu_k[:-1], cu_k[1:]):
        if b > a:
            o[a:b], lse[a:b], mag[a:b] = attend(q[a:b], k[c:e], v[c:e], scale,
                                                (e - c) - (b - a) if causal else None)
    return o, lse, mag


def gather(cache, table_row, n):
    page = cache.shape[1]
    t = np.arange(n)
    return cache[table_row[t // page], t % page]


def decode(q, k_cache, v_cache, table, lengths, scale):
    o, mag = np.empty(q.shape), np.empty(q.shape)
    lse = np.empty(q.shape[:2])
    for s, n in enumerate(lengths):
        o[s:s + 1], lse[s:s + 1], mag[s:s + 1] = attend(
            q[s:s + 1], gather(k_cache, table[s], n), gather(v_cache, table[s], n), scale)
    return o, lse, mag
