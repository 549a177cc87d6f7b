"""The check of cache_accuracy takes the arithmetic that the paged attention has, and none that lost a
part of it: emulated on the CPU, no GPU needed."""

import math

import numpy as np
import pytest

import cache_accuracy as A
import cache_reference as R


def _inputs(n, heads=16, seed=1):
    rng = np.random.default_rng(seed)
    x = R.VALUES[R.encode(rng.standard_normal((n, R.D)))]
    q = A._bf16(rng.standard_normal((heads, R.D)))
    s = q @ x.T / math.sqrt(R.D)
    m = s.max(axis=1, keepdims=True)
    p = np.exp(s - m)
    t = p.sum(axis=1, keepdims=True)
    p /= t
    return q, x, p @ x, (m + np.log(t))[:, 0], A.tolerance(p, x, np.ones(n), p @ x)


@pytest.mark.parametrize("n", [333, 20011])
def test_the_kernels_arithmetic_is_taken(n):
    q, x, ref, lse, tol = _inputs(n)
    o, l = A.emulate(q, x)
    A.check(o, ref, tol, l, lse)


@pytest.mark.parametrize("n", [333, 20011])
@pytest.mark.parametrize("lost", [dict(low_weights=False), dict(low_q=False), dict(skip=slice(128, 192))])
def test_a_lost_part_is_refused(n, lost):
    q, x, ref, lse, tol = _inputs(n)
    o, l = A.emulate(q, x, **lost)
    with pytest.raises(AssertionError, match="output is off"):
        A.check(o, ref, tol, l, lse)


def test_a_lost_tile_is_refused_by_lse_too():
    q, x, ref, lse, tol = _inputs(20011)
    _, l = A.emulate(q, x, skip=slice(19968, 20011))
    with pytest.raises(AssertionError, match="lse is off"):
        A.check(ref, ref, tol, l, lse)


def test_helpers_round_as_they_say():
    import torch
    y = np.concatenate([np.random.default_rng(2).standard_normal(4000) * np.exp2(np.arange(4000) % 30 - 18), [0.0]])
    t = torch.from_numpy(y)
    np.testing.assert_array_equal(A._bf16(y), t.float().to(torch.bfloat16).double().numpy())
    small = y.astype(np.float32).astype(np.float64)
    np.testing.assert_array_equal(A._e5m2(small), torch.from_numpy(small).float().to(torch.float8_e5m2).double().numpy())
