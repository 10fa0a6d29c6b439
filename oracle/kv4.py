"""fp64 oracle of the 4-bit key/value cache (numpy, no code shared with the GPU path).

A group of 64 values of a head's vector: z = fp16(min), a = fp16((max - min) /
15) with the difference and the quotient each rounded to fp32, code = (x - z) /
a to the nearest integer, halves to even, clamped to 0..15 (0 where a is 0),
standing for a code + z.  A group with a value that is not finite or beyond
+-60000 is NaN.  Positions are found through a page table; attention's softmax
runs over the positions that the masks leave.
"""
from __future__ import annotations

import numpy as np

GROUP = 64


def quantize(x):
    """x [..., D] -> (codes uint8 [..., D], param fp16 [..., D / 64, 2])."""
    x = np.asarray(x, dtype=np.float64)
    v = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    bad = ~(np.abs(v) <= 60000).all(-1)
    v = np.where(bad[..., None], 0.0, v)
    lo, hi = v.min(-1).astype(np.float32), v.max(-1).astype(np.float32)
    a = ((hi - lo) / np.float32(15)).astype(np.float16)
    z = lo.astype(np.float16)
    a64, z64 = a.astype(np.float64)[..., None], z.astype(np.float64)[..., None]
    code = np.rint((v - z64) / np.where(a64 > 0, a64, np.inf)).clip(0, 15).astype(np.uint8)
    param = np.stack([a, z], -1)
    param[bad] = np.nan
    return code.reshape(x.shape), param


def pack(code):
    """Codes [..., D] -> bytes [..., D / 2]: value 2b in the low bits of byte b."""
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)


def unpack(byte):
    out = np.empty((*byte.shape[:-1], 2 * byte.shape[-1]), dtype=np.uint8)
    out[..., 0::2], out[..., 1::2] = byte & 15, byte >> 4
    return out


def values(byte, param):
    """Bytes [..., D / 2] and param [..., D / 64, 2] -> values fp64 [..., D]."""
    code = unpack(byte).astype(np.float64)
    code = code.reshape(*code.shape[:-1], code.shape[-1] // GROUP, GROUP)
    p = param.astype(np.float64)
    return (code * p[..., :1] + p[..., 1:]).reshape(*byte.shape[:-1], 2 * byte.shape[-1])


def magnitudes(byte, param):
    """a code + |z|: what the roundings of a value and of its parts scale with."""
    code = unpack(byte).astype(np.float64)
    code = code.reshape(*code.shape[:-1], code.shape[-1] // GROUP, GROUP)
    p = param.astype(np.float64)
    return (code * p[..., :1] + np.abs(p[..., 1:])).reshape(*byte.shape[:-1], 2 * byte.shape[-1])


def gather(array, table_row, n):
    """Positions 0..n-1 of one sequence from [pages][heads][page_size][...]:
    [n][heads][...]."""
    page_size = array.shape[2]
    at = np.arange(n)
    return array[np.asarray(table_row)[at // page_size], :, at % page_size]


def visible(n, new, i, causal=True, window=0):
    """Positions that row i of `new` rows sees in a sequence of n: a mask [n]."""
    pos = n - new + i
    at = np.arange(n)
    see = np.ones(n, dtype=bool)
    if causal:
        see &= at <= pos
    if window > 0:
        see &= at > pos - window
    return see


def attention(q, k, kp, v, vp, table, kv_len, cu, scale, causal=True, window=0, hidden=()):
    """q [T][H][D]; the cache's arrays; returns (out, lse, mag): fp64 [T][H][D],
    [T][H], and a dict of the sums that tolerances are made of -- "v": sum_j p_j
    (a code + |z|)_j of V [T][H][D], "s": the largest |scale| sum_d |q_d| (a
    code + |z|)_d of K over a row's positions [T][H].  Rows of no sequence are NaN.  hidden: positions that no
    row sees."""
    q = np.asarray(q, dtype=np.float64)
    T, H, D = q.shape
    heads = k.shape[1]
    out, lse = np.full((T, H, D), np.nan), np.full((T, H), np.nan)
    mag = {"v": np.zeros((T, H, D)), "s": np.zeros((T, H))}
    for b, n in enumerate(kv_len):
        K, V = (values(gather(x, table[b], n), gather(p, table[b], n)) for x, p in ((k, kp), (v, vp)))
        Km, Vm = (magnitudes(gather(x, table[b], n), gather(p, table[b], n))
                  for x, p in ((k, kp), (v, vp)))
        new = cu[b + 1] - cu[b]
        for i in range(new):
            t = cu[b] + i
            see = visible(n, new, i, causal, window)
            see[[j for j in hidden if j < n]] = False
            for h in range(H):
                g = h // (H // heads)
                out[t, h], lse[t, h] = 0.0, -np.inf
                if not see.any():
                    continue
                s = scale * (K[see, g] @ q[t, h])
                top = s.max()
                e = np.exp(s - top)
                p = e / e.sum()
                out[t, h] = p @ V[see, g]
                lse[t, h] = top + np.log(e.sum())
                mag["v"][t, h] = p @ Vm[see, g]
                mag["s"][t, h] = (abs(scale) * (Km[see, g] @ np.abs(q[t, h]))).max()
    return out, lse, mag
