"""Plain 64-bit forms of the 8-bit serving operators (W8A8 product, paged 8-bit
key/value cache, attention over it) for the GPU tests, in numpy.  Quantiser
decisions are defined in IEEE fp32 and taken in numpy's fp32."""
from __future__ import annotations

import numpy as np


def quantize_rows(x):
    """(codes int8, scales fp32) per row: s = fp32(amax / 127), 1 for a zero row; NaN and zero codes for a row that
    holds an infinity or a NaN."""
    x = np.asarray(x, dtype=np.float32)
    finite = np.isfinite(x).all(axis=1)
    amax = np.where(finite, np.abs(np.where(np.isfinite(x), x, 0)).max(axis=1), 0).astype(np.float32)
    s = np.where(amax > 0, amax / np.float32(127), np.float32(1)).astype(np.float32)
    q = np.clip(np.rint(np.where(finite[:, None], x, 0) / s[:, None]), -127, 127).astype(np.int8)
    return q, np.where(finite, s, np.float32(np.nan)).astype(np.float32)


def w8a8(X, mods, B):
    """X fp16 (T x d); mods: [(codes, scales, A or None)]; B (r x d) or None.
    Returns ([(y, bound)], (R, bound)): exact values and how far a correct kernel may be from each."""
    codes, st = quantize_rows(X)
    X64 = X.astype(np.float64)
    d = X.shape[1]
    u16, u32 = 2.0 ** -11, 2.0 ** -23          # half a step of fp16; a step of fp32 (sums may truncate)
    R = Rb = None
    if B is not None:
        B64 = B.astype(np.float64)
        R = X64 @ B64.T
        # R: one rounding to fp16 of an fp32 sum of d products (each term takes part in at most d additions)
        Rb = u16 * np.abs(R) + d * u32 * (np.abs(X64) @ np.abs(B64).T) + 2.0 ** -25
    out = []
    for q, s, A in mods:
        base = (codes.astype(np.float64) @ q.astype(np.float64).T) * st[:, None].astype(np.float64) * s.astype(np.float64)
        y, b = base, 4 * u32 * np.abs(base)    # int -> fp32, two products, one sum
        if A is not None and R is not None:
            A64 = np.abs(A.astype(np.float64))
            y = base + R @ A.astype(np.float64).T
            b = b + Rb @ A64.T + (A.shape[1] + 1) * u32 * (np.abs(R) @ A64.T)
        out.append((y, b + u16 * (np.abs(y) + b) + 2.0 ** -25))
    return out, (R, Rb)


def within(got, ref, bound):
    """Largest error in units of its bound (<= 1 passes); NaN must meet NaN."""
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == ref.shape, (got.shape, ref.shape)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    ok = ~np.isnan(ref)
    return float(np.max(np.abs(got - ref)[ok] / bound[ok], initial=0.0))
