"""GPU tests of how near the paged attention comes to 64 bits, relative to its own output
(cache_accuracy), where the elementwise bounds of cache_reference are wide."""

import math

import numpy as np
import pytest
import torch

import cache_accuracy as A
import cache_reference as R
from gpu_helpers import to_f64
from test_gpu_cache import DEV, Pool, _i32, _smla, bf16, bf16_dev

pytestmark = pytest.mark.gpu


def _attend(pool, table, lens, q, **kw):
    o, lse = _smla().sparse_mla_fwd_paged(bf16_dev(q), pool.device(), _i32(table), _i32(lens),
                                          **{k: _i32(v) for k, v in kw.items()})
    return to_f64(o), lse.double().cpu().numpy()


@pytest.mark.parametrize("H", [16, 64, 128])
@pytest.mark.parametrize("lens", [[333, 700, 4097], [20011]])
def test_flat_weights(H, lens):
    pool = Pool(sum(-(-n // 64) for n in lens) + 1, 64, 64, seed=90, junk=False)
    table = pool.place(lens)
    pool.fill(table, lens)
    q = bf16(np.random.default_rng(H).standard_normal((len(lens), H, 512)))
    o, lse = _attend(pool, table, lens, q)
    at = (q, pool.codes, pool.scales, table, lens, 64, 64)
    ref, rl, _, _ = R.attend(*at)
    A.check(o, ref, A.tolerances(*at), lse, rl)


@pytest.mark.parametrize("H,K", [(32, 400), (128, 512)])
def test_flat_weights_of_picks(H, K):
    rng = np.random.default_rng(K)
    pool = Pool(60, 64, 32, seed=91, junk=False)
    lens = [3000, 600]
    table = pool.place(lens)
    pool.fill(table, lens)
    seq = np.arange(40) % 2
    ln = np.array(lens)[seq]
    topk = np.stack([rng.permutation(n)[:K] for n in ln])
    q = bf16(rng.standard_normal((40, H, 512)))
    o, lse = _attend(pool, table, ln, q, topk=topk, seq=seq)
    at = (q, pool.codes, pool.scales, table, ln, 64, 32, topk, seq)
    ref, rl, _, _ = R.attend(*at)
    A.check(o, ref, A.tolerances(*at), lse, rl)


def test_every_tile_of_a_split_sequence_counts():
    # a head for each tile of 64, drawn to one row of it by some 14 nats: a tile that is lost or
    # taken twice is the whole output of its head
    n, H = 20011, 128
    rng = np.random.default_rng(92)
    pool = Pool(314, 64, 64, seed=93, junk=False)
    table = pool.place([n])
    pool.fill(table, [n])
    at = np.minimum(np.arange(3 * H) % 313 * 64 + rng.integers(0, 64, size=3 * H), n - 1)
    x, _, _ = R.rows_of(pool.codes, pool.scales, table[0], at, 64, 64)
    q = bf16(x.reshape(3, H, 512) * (14 * math.sqrt(512) / 512))
    o, lse = _attend(pool, table, [n] * 3, q, seq=[0, 0, 0])
    at = (q, pool.codes, pool.scales, table, [n] * 3, 64, 64, None, [0, 0, 0])
    ref, rl, _, _ = R.attend(*at)
    A.check(o, ref, A.tolerances(*at), lse, rl)


# One token repeated: as many tokens as CTAs, so that a CTA has one token's tiles in a run.
def _repeated(pool, table, n, q, topk=None):
    T = 160
    kw = {} if topk is None else dict(topk=np.repeat(topk[None], T, 0))
    o, lse = _attend(pool, np.asarray(table), [n] * T, np.repeat(q, T, 0), seq=np.zeros(T), **kw)
    at = (q, pool.codes, pool.scales, table, [n], pool.page, pool.block, None if topk is None else topk[None])
    ref, rl, _, _ = R.attend(*at)
    return o, lse, ref, rl, A.tolerances(*at)


def _loud(rng, n, louder):
    """Rows of N(0,1), the first one `louder` times as loud and turned away from all heads; q."""
    q = bf16(rng.standard_normal((1, 16, 512)))
    rows = rng.standard_normal((n, 512))
    rows[0] = -q[0].sum(axis=0) / 4 * louder
    pool = Pool(-(-n // 64), 64, 16, seed=94, junk=False)
    table = pool.place([n])
    R.write(pool.codes, pool.scales, table, [0], [0, n], bf16(rows), 64, 16)
    return pool, table, q


def test_a_loud_row_that_nobody_heeds():
    # its block's scale is 2^14 that of the others, its weight nothing: the others' weights must
    # not lose its scale's range (a part of a token has its own largest weight: one tolerance holds for all)
    rng = np.random.default_rng(95)
    pool, table, q = _loud(rng, 4096, 2.0 ** 14)
    picks = np.concatenate([[0], 16 + rng.permutation(4080)[:511]])       # none of its block's other rows
    o, lse, ref, rl, tol = _repeated(pool, table, 4096, q, picks)
    A.check(o, ref, tol, lse, rl)


def test_a_loud_block_in_ordinary_company():
    # all of the block's rows have the loud row's scale, and scores like any other: they take 2^12 of the weights'
    # range. What is off by 2^-20 of the largest weight is then 2^-8 of theirs at most.
    pool, table, q = _loud(np.random.default_rng(96), 512, 2.0 ** 12)
    o, lse, ref, rl, tol = _repeated(pool, table, 512, q)
    A.check(o, ref, tol, lse, rl)


@pytest.mark.parametrize("n", [8192, 32768])
@pytest.mark.parametrize("spread", [0.1, 0.3, 1.0])
def test_one_row_against_thousands(n, spread):
    # the first row has half of the weight (as a first token often has), thousands of nearly equal ones
    # with a common direction the other half: their weights are 2^-13 and 2^-15 of the largest. They are held
    # to 2^-20 of it, that is 2^-7 and 2^-5 of themselves; spread over more than such a step (a
    # tenth of a nat is 2^-2.8 of them) they have no common sign for more than a quarter of it:
    # 2^-7 of half the output at most, beside the output's own rounding, 1.7e-3.
    rng = np.random.default_rng(n)
    d = rng.standard_normal(512)
    d /= np.linalg.norm(d)

    def apart(v):
        return v - (v @ d)[..., None] * d
    rows = apart(rng.standard_normal((n, 512)) * 0.5) + 0.5 * apart(rng.standard_normal(512))
    rows += spread * rng.standard_normal((n, 1)) * d                     # scores of N(0, spread)
    rows[0] = apart(rng.standard_normal(512) * 0.5) + (math.log(n) + spread ** 2 / 2) * d
    q = bf16((math.sqrt(512) * d + 0.02 * spread * rng.standard_normal((1, 16, 512))))
    pool = Pool(n // 64, 64, 64, seed=97, junk=False)
    table = pool.place([n])
    R.write(pool.codes, pool.scales, table, [0], [0, n], bf16(rows), 64, 64)
    o, lse, ref, rl, _ = _repeated(pool, table, n, q)
    A.check(o, ref, math.hypot(1.7e-3, 2.0 ** -8) * np.linalg.norm(ref, axis=-1), lse, rl)
