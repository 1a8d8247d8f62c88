"""fp64 definitions (numpy) of paged attention, of the cache's codes and of the
verification of drafts, with the bounds that the kernels' roundings allow."""
from __future__ import annotations

import numpy as np

BF16 = 2.0 ** -8   # one rounding to bf16, relative
FP16 = 2.0 ** -11  # one rounding to fp16, relative
LEAST = 2.0 ** -126


def scales(x, kv):
    """The scales [..] (float32) of rows x [.., D] (exact bf16 values)."""
    top = np.abs(np.asarray(x, np.float64)).max(-1)
    with np.errstate(invalid="ignore"):
        if kv == "int8":
            s = np.maximum((top / 127).astype(np.float32).astype(np.float64), LEAST)
        else:
            m, e = np.frexp(top / 448)  # top / 448 = m 2^e, 1/2 <= m < 1
            s = np.where(top > 0, np.ldexp(1.0, np.where(m == 0.5, e - 1, e)), LEAST)
            s = np.maximum(s, LEAST)
    return np.where(np.isfinite(top), s, np.nan).astype(np.float32)


def codes(x, s, kv):
    """What the codes stand for without their scale (0 in rows of scale NaN)."""
    with np.errstate(invalid="ignore"):
        y = np.asarray(x, np.float64) / s.astype(np.float64)[..., None]
        if kv == "int8":
            c = np.rint(y)
        else:  # steps of 1/8 of the value's power of two, none below 2^-9
            ulp = np.ldexp(1.0, np.maximum(np.frexp(np.abs(y))[1] - 1, -6) - 3)
            c = np.rint(y / ulp) * ulp
    return np.where(np.isfinite(s)[..., None], c, 0.0)


def attention(q, k, v, length, scale, window, k_scale=None, v_scale=None):
    """One sequence: q [n][Hq][D] at its last positions, k, v [length][Hkv][D],
    for an 8-bit cache their scales [length][Hkv].  Returns out and, per output,
    how far off it may be."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    n, g = q.shape[0], q.shape[1] // k.shape[1]
    at, key = length - n + np.arange(n)[:, None], np.arange(length)[None]
    seen = (key <= at) & (key > at - window if window else True)
    codes_wide = v_scale is not None and n * g > 16  # the tensor cores' kernel
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    for h in range(q.shape[1]):
        kk, vv = k[:, h // g], v[:, h // g]
        s = np.where(seen, q[:, h] @ kk.T * scale, -np.inf)
        w = np.exp(s - s.max(1, keepdims=True))
        w /= w.sum(1, keepdims=True)
        o, mass = w @ vv, w @ np.abs(vv)
        terms = np.where(seen, np.abs(q[:, h]) @ np.abs(kk).T, 0.0).max(1, keepdims=True) * abs(scale)
        # A score in fp32 is off by 2^-21 of its terms' sum (sums in any order, the
        # products by the scales and by log2 e, the difference to the maximum).
        slip = 2.0 ** -21 * terms
        weight = BF16 if v_scale is None else FP16
        floor = 3 * 2.0 ** -126 * (seen @ np.abs(vv))
        if v_scale is not None:
            kt, vt = (np.abs(x[:, h // g].astype(np.float64)) for x in (k_scale, v_scale))
            if codes_wide:
                # Each value of k is one fp16 rounding off: the sum of D independent
                # ones lies within 8 standard deviations, of 2^-11 / sqrt(3) of the
                # root of the terms' squares.  Scales under a power of two that brings
                # the key tile's largest to 2^5 or more are two fp16 terms, off by
                # 2^-26: a code of at most 448 by 2^-22 of the largest scale.
                square = np.where(seen, (q[:, h] ** 2) @ (kk ** 2).T, 0.0).max(1, keepdims=True)
                slip = slip + 8 * FP16 / 3 ** 0.5 * np.sqrt(square) * abs(scale)
                slip = slip + 2.0 ** -22 * np.abs(q[:, h]).sum(1, keepdims=True) * kt.max() * abs(scale)
                # A value of v is two fp16 roundings off (its scale's and its own), and
                # 2^-21 of the largest scale so far (a scale's step at 2^-14 below 2^5, times
                # 448); a weight's fp16 is of 2^7 times it: off by 2^-32 at most.
                weight = 3 * FP16
                floor = floor + 2.0 ** -21 * vt.max() + 2.0 ** -32 * (seen @ np.abs(vv))
            else:
                # A product t of a weight and a scale enters as fp16 of t 2^7 / r, r a
                # power of two at or below the row's largest t: fp16 has steps of 2^-24
                # below 2^-14, so that each t is off by at most 2^-25 / 2^7 r <= 2^-32 of
                # the largest, whatever its size, and each term by that times its code.
                floor = floor + 2.0 ** -32 * (w * vt).max(1, keepdims=True) * (
                    seen @ np.abs(vv / vt[:, None]))
        # Two factors of 2^slip (a weight and the weights' total); the exponentials
        # and the sums over the keys are off by 2^-18 at most.  Weights are fp32
        # beside the largest one's 1: below 2^-126 they count as 0, and so do the
        # factors that bring a part's sums (of terms of at most |v| each) to another
        # maximum, within the keys, between warps and between blocks.
        slip = np.expm1(2 * slip)
        out[:, h] = o
        bound[:, h] = BF16 * np.abs(o) + (weight + 2.0 ** -18 + slip) * mass + floor + 1e-37
    return out, bound


def verify(target, draft, drafted, uniform):
    """One sequence: target [T + 1][V], draft [T][V] or None, drafted [T],
    uniform [T + 1] (float32 values).  Returns (accepted, the token after them,
    the running sums and the aim that chose it)."""
    T, V = len(drafted), target.shape[1]
    a = 0
    while a < T and drafted[a] >= 0:
        q = 1.0 if draft is None else float(draft[a, drafted[a]])
        if not float(uniform[a]) * q < float(target[a, drafted[a]]):
            break
        a += 1
    w = target[a].astype(np.float64)
    if a < T and drafted[a] >= 0:
        if draft is None:
            less = np.zeros(V)
            less[drafted[a]] = 1.0
        else:
            less = draft[a].astype(np.float64)
        rest = np.maximum(w - less, 0.0)
        if rest.sum() > 0:
            w = rest
    cum = np.cumsum(w)
    aim = float(uniform[T]) * cum[-1]
    token = int(np.searchsorted(cum, aim, side="right"))
    if token == V:  # the aim rounded up to the total
        token = int(np.nonzero(w)[0][-1])
    return a, token, cum, aim
