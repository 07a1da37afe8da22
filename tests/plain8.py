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


# ------------------------------------------------------- key/value cache ----

PAGE = 64


def rope_table(positions, D, theta=10000.0):
    """Cosines of the D/2 pairs, then sines, by position (fp32)."""
    inv = theta ** (-np.arange(0, D, 2) / D)
    ang = np.arange(positions)[:, None] * inv
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def rotate(x, cs):
    """x (n x heads x D fp16), cs (n x D fp32): two fp32 products and a sum, unfused, rounded to fp16 -- the
    operator's definition, so stored values can be compared bit by bit."""
    half = x.shape[-1] // 2
    a, b = x[..., :half].astype(np.float32), x[..., half:].astype(np.float32)
    c, s = cs[:, None, :half], cs[:, None, half:]
    with np.errstate(over="ignore", invalid="ignore"):
        return np.concatenate([(a * c - b * s).astype(np.float16), (b * c + a * s).astype(np.float16)], -1)


def quantize_page(x):
    """One page and head (64 x D fp16) -> (codes, scale)."""
    x = x.astype(np.float32)
    if not np.isfinite(x).all():
        return np.zeros(x.shape, np.int8), np.float32(np.nan)
    s = np.float32(max(np.abs(x).max(), np.float32(2.0 ** -24))) / np.float32(127)
    return np.clip(np.rint(x / s), -127, 127).astype(np.int8), s


class Sequence:
    """The keys and values of one sequence as the cache defines them: fp16 (keys rotated), whole pages quantised."""

    def __init__(self, H, D):
        self.k, self.v = np.zeros((0, H, D), np.float16), np.zeros((0, H, D), np.float16)

    def append(self, k, v):
        self.k, self.v = np.concatenate([self.k, k]), np.concatenate([self.v, v])

    def held(self):
        """(keys, values) in 64 bits, len x H x D."""
        out = []
        for x in (self.k, self.v):
            y = x.astype(np.float64)
            for p in range(len(x) // PAGE):
                for h in range(x.shape[1]):
                    q, s = quantize_page(x[p * PAGE:(p + 1) * PAGE, h])
                    y[p * PAGE:(p + 1) * PAGE, h] = q.astype(np.float64) * np.float64(s)
            out.append(y)
        return out


def attention(Q, k, v, start, scale):
    """Q (n x Hq x D fp16) at positions start .. over k, v (len x H x D, 64 bits).  Returns (Y, bound)."""
    n, Hq, D = Q.shape
    L, H = k.shape[:2]
    G = Hq // H
    Y, bound = np.zeros((n, Hq, D)), np.full((n, Hq, D), 2.0 ** -25)
    u16, u32 = 2.0 ** -11, 2.0 ** -23
    for i in range(n):
        m = min(L, start + i + 1)
        if m <= 0:
            continue
        for h in range(Hq):
            with np.errstate(over="ignore", invalid="ignore"):
                q, kk, vv = Q[i, h].astype(np.float64), k[:m, h // G], v[:m, h // G]
                s = kk @ q * scale
                w = np.exp(s - s.max())
                p = w / w.sum()
                y = p @ vv
                # fp32 scores: D products summed, the scales and log2 e applied, in a range of |s| and of the maximum's
                ds = (D + 6) * u32 * (np.abs(kk) @ np.abs(q)) * scale + 4 * u32 * (np.abs(s) + abs(s.max()))
                # weights: that error in the exponent, exp2's own (2^-22), fp16 rounding; below fp16's normals an absolute 2^-33
                dw = 2 * ds + 2.0 ** -22 + u16
                # sums over m terms in fp32: each weight and product, and the rescalings of one per page
                acc = (m + 8) * u32
                spread = p @ (np.abs(vv) * (dw[:, None] + acc)) + np.abs(y) * (p @ (dw - u16) + acc)
                # a weight below fp16's normals is off by 2^-33 of the largest weighted value's unit, and values
                # are at most 128 units of their page (64 .. 128 in a tail)
                spread += 2.0 ** -33 * 2 * m * np.abs(vv).max(initial=0.0) / w.sum()
            Y[i, h] = y
            bound[i, h] += spread + u16 * (np.abs(y) + spread)
    return Y, bound
