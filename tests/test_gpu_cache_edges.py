"""GPU tests of the paged 8-bit cache's attention at the edges of its inputs: queries that are not
finite or near the end of bf16's range, and tokens that see nothing.

Models, bounds and the pool are those of test_gpu_cache.
"""

import math

import numpy as np
import pytest
import torch

import cache_reference as R
from gpu_helpers import to_f64
from test_gpu_cache import DEV, Pool, _attend_and_check, _i32, _smla, bf16

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K", [0, 40, 900])
@pytest.mark.parametrize("H", [16, 80])
def test_tokens_that_see_nothing_are_zero_whatever_q_holds(H, K):
    # padded slots and tokens without a valid pick (K 900: split over several CTAs), whose q is
    # infinite or NaN: o = 0 and lse = sink; a token that sees one row is NaN in the heads concerned
    smla = _smla()
    rng = np.random.default_rng(K + H)
    pool = Pool(40, 16, 16, seed=80)
    table = pool.place([100, 230])
    pool.fill(table, [100, 230])
    cache = pool.device()
    seq = np.array([0, 0, 1, 1, 0, 1])
    lens = np.array([0, 0, 0, 0, 100, 1])
    q = rng.standard_normal((6, H, 512))
    q[0], q[1], q[2, :, 7], q[3, ::2, 500] = np.nan, np.inf, -np.inf, np.nan
    q[4, 3, 11], q[5, 5, 400], q[5, 6, 1] = np.inf, -np.inf, np.nan
    topk = None
    if K:
        lens[2:4] = 230                                  # these see rows, but pick none
        topk = rng.integers(0, 100, size=(6, K))
        topk[:4] = -1
        topk[5] = -1
        topk[5, K // 2] = 0
    sink = rng.standard_normal(H).astype(np.float32)
    qd = torch.from_numpy(q).to(torch.bfloat16).to(DEV)
    for with_sink in (True, False):
        o, lse = smla.sparse_mla_fwd_paged(qd, cache, _i32(table), _i32(lens), seq=_i32(seq),
                                           topk=None if topk is None else _i32(topk),
                                           sink=torch.from_numpy(sink).to(DEV) if with_sink else None)
        o, lse = to_f64(o), lse.double().cpu().numpy()
        assert (o[:4] == 0).all()
        if with_sink:
            # log2(e) and back, and a sum of one: four roundings of 2^-24
            assert (np.abs(lse[:4] - sink) <= 2.0 ** -22 * np.abs(sink)).all()
        else:
            assert np.isneginf(lse[:4]).all()
        nan = np.zeros((2, H), dtype=bool)
        nan[0, 3] = nan[1, 5] = nan[1, 6] = True
        assert np.isnan(o[4:][nan]).all() and np.isnan(lse[4:][nan]).all()
        assert np.isfinite(o[4:][~nan]).all() and np.isfinite(lse[4:][~nan]).all()


@pytest.mark.parametrize("K", [0, 70])
def test_q_up_to_the_largest_bf16(K):
    # rows of q whose largest value is 1.75 * 2^127 and above, up to bf16's largest; rows of the cache and the score
    # scale are small, so that scores are ordinary
    rng = np.random.default_rng(81)
    lens = [150, 70, 9]
    pool = Pool(30, 16, 16, seed=82)
    table = pool.place(lens)
    pool.fill(table, lens, amp=2.0 ** -60)
    q = np.clip(rng.standard_normal((3, 32, 512)), -3, 3) * 2.0 ** 125
    for h in range(32):
        big = (1.75 + 2.0 ** -7 * (h % 32)) * 2.0 ** 127             # 1.75, ..., 1.9921875, the largest
        q[:, h, rng.integers(0, 512)] = min(big, 1.9921875 * 2.0 ** 127) * (-1) ** h
    topk = rng.integers(0, np.array(lens)[:, None], size=(3, K)) if K else None
    # |q . x| is about 2^(126 - 60) * 22, times 2^-70: scores of order one
    _attend_and_check(pool, table, lens, 32, seed=83, q=q, topk=topk, scale=2.0 ** -70)


@pytest.mark.parametrize("K", [0, 5])
def test_scores_past_float_leave_masked_tokens_alone(K):
    # q and the score scale are finite, their product is not: a token that sees nothing is zero all the same
    smla = _smla()
    pool = Pool(4, 16, 16, seed=84)
    table = pool.place([20])
    pool.fill(table, [20])
    q = torch.full((2, 16, 512), 3e38, dtype=torch.bfloat16, device=DEV)
    topk = torch.full((2, K), -1, dtype=torch.int32, device=DEV) if K else None
    o, lse = smla.sparse_mla_fwd_paged(q, pool.device(), _i32(table), _i32([20, 0] if K else [0, 0]), topk=topk,
                                       seq=_i32([0, 0]), scale=1e10)
    assert (o == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("T", [1, 160])                      # split over eight CTAs; several tokens a CTA
@pytest.mark.parametrize("at", [0, 250, 511])
def test_a_row_near_the_end_of_the_range_leaves_the_sums_alone(T, at):
    # one row 2^130 times the others, turned away from all heads: the other fifteen rows of its block are zeros at its
    # scale, and count in the denominator like the 496 ordinary rows, whose outputs they drown
    rng = np.random.default_rng(85)
    n = 512
    q = bf16(rng.standard_normal((160, 16, 512)))
    q[1:] = q[0]
    rows = rng.standard_normal((n, 512)) * 2.0 ** -20
    rows[at] = -q[0].sum(axis=0) / 4 * 2.0 ** 110
    pool = Pool(n // 64, 64, 16, seed=86, junk=False)
    table = pool.place([n])
    R.write(pool.codes, pool.scales, table, [0], [0, n], bf16(rows), 64, 16)
    o, lse = _smla().sparse_mla_fwd_paged(torch.from_numpy(q[:T]).to(torch.bfloat16).to(DEV), pool.device(), _i32(table),
                                          _i32([n] * T), seq=_i32(np.zeros(T)))
    _, rl, _, _ = R.attend(q[:1], pool.codes, pool.scales, table, [n], 64, 16)
    # 511 scores of next to nothing: lse is log(511) to a few roundings of its sum and of a logarithm of 2^116 (each 2^-24
    # of 81 nats)
    assert np.abs(rl - np.log(511)).max() < 1e-4
    assert np.abs(lse.double().cpu().numpy() - rl).max() <= 511 * 2.0 ** -23 + 4 * 81 * 2.0 ** -23
    assert torch.isfinite(o).all()


def test_rows_of_zeros_count_beside_loud_ones():
    # rows of zeros have the least scale, 2^-100: 16,000 of them beside one row of scale 2^13 that every head
    # gives 2^22 times the weight of a zero row
    rng = np.random.default_rng(87)
    n = 16016
    d = rng.standard_normal(512)
    d /= np.linalg.norm(d)
    q = bf16(math.sqrt(512) * 2.0 ** -20 * (d + 1e-3 * rng.standard_normal((160, 16, 512))))
    q[1:] = q[0]
    rows = np.zeros((n, 512))
    rows[n - 3] = 22 * math.log(2.0) * 2.0 ** 20 * d
    for first in (False, True):
        pool = Pool(-(-n // 64), 64, 16, seed=88, junk=False)
        table = pool.place([n])
        R.write(pool.codes, pool.scales, table, [0], [0, n], bf16(rows[::-1] if first else rows), 64, 16)
        assert pool.scales.max() >= 2.0 ** 8 and pool.scales.min() == 2.0 ** -100
        o, lse = _smla().sparse_mla_fwd_paged(torch.from_numpy(q).to(torch.bfloat16).to(DEV), pool.device(),
                                              _i32(table), _i32([n] * 160), seq=_i32(np.zeros(160)))
        ref, rl, _, _ = R.attend(q[:1], pool.codes, pool.scales, table, [n], 64, 16)
        # without the rows of zeros lse would be log(1 + 16,000 / 2^22) = 4e-3 less; their sum's roundings are
        # 16,000 * 2^-24 of that, lse's of 15 nats, and the score's 512 * 2^-23 of 15
        assert np.abs(lse.double().cpu().numpy() - rl).max() <= 16000 * 2.0 ** -24 * 4e-3 + 15 * 520 * 2.0 ** -23
        worst = np.linalg.norm(to_f64(o) - ref, axis=-1) / np.linalg.norm(ref, axis=-1)
        assert worst.max() <= 2.0 ** -8 + 1e-3
