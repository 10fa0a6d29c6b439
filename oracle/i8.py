"""fp64 oracle of the 8-bit integer product (numpy, no code shared with the GPU path).

quantize: with a = max_k |x[m][k]|, code = 127 x / a rounded to the nearest
integer, halves to even; scale = a / 127 rounded to fp32.  The quotient is
taken in fp64 after an exact product: 127 x of an fp16 or bf16 x has at most 18
significant bits and a at most 11, so a quotient that is no half of an integer
differs from one by more than fp64's rounding.
gemm: the exact integer sum times the two scales.
"""
from __future__ import annotations

import numpy as np


def quantize(x):
    """x [M][K] (values of a 16-bit type, any float dtype) -> (codes int8, scale fp32)."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(x).max(axis=1)
    bad = ~np.isfinite(x).all(axis=1)
    scale = (a.astype(np.float32) / np.float32(127)).astype(np.float32)
    scale[bad] = np.nan
    ok = (a > 0) & ~bad
    q = np.zeros(x.shape, dtype=np.int8)
    q[ok] = np.rint(127.0 * x[ok] / a[ok, None]).astype(np.int8)
    return q, scale


def gemm(x, sx, w, sw):
    """Codes int8 [M][K], [N][K] and scales -> y fp64 [M][N]."""
    acc = np.asarray(x, dtype=np.int64) @ np.asarray(w, dtype=np.int64).T
    return acc * np.asarray(sx, np.float64)[:, None] * np.asarray(sw, np.float64)[None, :]
