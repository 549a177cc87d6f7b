"""Errors of the paged attention relative to its output, head by head, and an emulation of its
arithmetic (numpy, on the CPU) for tests of that check.

cache_reference.attend's bound adds every rank's worst rounding with one sign: it grows with the sum of the weights
times |x|, while |o| of many independent rows shrinks. Here the error's norm over a head's 512 outputs is held
against what roundings without a common sign add up to:
* the output's rounding to bf16: at most 2^-8 of a value, spread evenly over that step: 2^-8 / sqrt(3) of the step's
  lower end, 1.66e-3 of the norm for values of every size (the mean square of 1/m, m even in its logarithm over [1, 2),
  is 0.54). Over 512 outputs, of which the larger ones count, it spreads by some 3%: 2e-3 is five times that above;
* a weight p, held as an e4m3 part and an e5m2 part of the rest, is off by at most 2^-7 of it, or by 2^-20 of the
  largest weight where weights count with their blocks' scales (include/smla.h): e. In the mean square it is
  1.4e-3 of it (the rest 2^-4 / sqrt(3) * 0.74, its rounding 2^-3 / sqrt(3) * 0.74 of that), so sqrt(sum e^2 |x|^2), the
  square root of the worst cases' squares, is 5.5 standard deviations of their sum, and the very bound where one rank
  has nearly all;
* scores: an fp32 sum of 512 products whose partial sums stay below 4 sqrt(512) for q and x of N(0,1), off by at most
  512 * 4 sqrt(512) * 2^-23 / sqrt(512) = 2.5e-4 nats even if each addition truncates; a common shift leaves o alone.
LSE_TOL is twice the scores' bound (sums of n positive terms in fp32 add 6 sqrt(n) 2^-24 at most in practice, 5e-5 for
20,000).
"""

from __future__ import annotations

import math

import numpy as np

import cache_reference as R

LSE_TOL = 5e-4


def tolerance(p, x, scales, o):
    """What a head's output may be off by, [H]: weights p [H,n], rows x [n,512] and their block scales [n], o [H,512]."""
    unit = 2.0 ** -20 * (p * scales).max(axis=1, keepdims=True) / scales
    e = np.maximum(2.0 ** -7 * p, unit)
    return np.hypot(2e-3 * np.linalg.norm(o, axis=1), np.linalg.norm(e * np.linalg.norm(x, axis=1), axis=1))


def tolerances(q, codes, scales, table, lens, page, block, topk=None, seq=None):
    """tolerance [T,H] of the tokens of cache_reference.attend (no sink, the default score scale)."""
    out = np.zeros(q.shape[:2])
    for t in range(len(q)):
        pos = np.arange(lens[t]) if topk is None else topk[t][topk[t] >= 0]
        x, sc, _ = R.rows_of(codes, scales, table[t if seq is None else int(seq[t])], pos.astype(np.int64), page, block)
        s = q[t] @ x.T / math.sqrt(R.D)
        p = np.exp(s - s.max(axis=1, keepdims=True))
        p /= p.sum(axis=1, keepdims=True)
        out[t] = tolerance(p, x, sc, p @ x)
    return out


def check(got, ref, tol, lse=None, ref_lse=None):
    """Raises AssertionError if a head's output (its norm over the last axis) or lse is further off."""
    err = np.linalg.norm(got - ref, axis=-1)
    over = (err / tol).max()
    assert over <= 1, f"a head's output is off by {(err / np.linalg.norm(ref, axis=-1)).max():.2e} of its norm, " \
                      f"{over:.2f} of what it may be"
    if lse is not None:
        d = float(np.abs(lse - ref_lse).max())
        assert d <= LSE_TOL, f"lse is off by {d:.2e}, more than {LSE_TOL:.1e}"


def _e5m2(y):
    """The e5m2 values nearest to y (ties to even; |y| below 2^15)."""
    e = np.maximum(np.frexp(np.abs(y))[1] - 1, -14)
    return np.ldexp(np.rint(np.ldexp(y, 2 - e)), e - 2)


def _bf16(y):
    f = np.asarray(y, dtype=np.float32).view(np.uint32).astype(np.uint64)
    f = (f + 0x7FFF + ((f >> 16) & 1)) & 0xFFFF0000
    return f.astype(np.uint32).view(np.float32).astype(np.float64)


def emulate(q, x, low_weights=True, low_q=True, skip=None):
    """(o [H,512] rounded to bf16, lse [H]) of rows x [n,512] (a block scale of 1) as the kernel holds q and the
    weights: e4m3 and what is left of it. The parts can be left out, and so can the ranks of `skip` (a slice)."""
    scale = np.exp2(np.ceil(np.log2(np.abs(q).max(axis=1, keepdims=True) / 448.0)))
    y = q / scale
    hi = R.VALUES[R.encode(y)]
    if low_q:
        hi = hi + R.VALUES[R.encode(16.0 * (y - hi))] / 16.0
    s = hi * scale @ x.T / math.sqrt(R.D)
    if skip is not None:
        s[:, skip] = -np.inf
    m = s.max(axis=1, keepdims=True)
    p = np.exp(s - m)
    w = R.VALUES[R.encode(16.0 * p)]
    if low_weights:
        w = w + _e5m2(16.0 * p - w)
    total = p.sum(axis=1, keepdims=True)
    return _bf16((w / 16.0) @ x / total), (m + np.log(total))[:, 0]
