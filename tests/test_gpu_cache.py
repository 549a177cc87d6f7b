"""GPU tests of the paged 8-bit cache: row writes, page management and the
attention over it, each against the 64-bit models of cache_reference.

Codes, scales, tables and counts are compared exactly (a scale is a power of
two, so every code is the rounding of an exact quotient); the attention's
outputs within the bounds derived in cache_reference.attend.
"""

import numpy as np
import pytest
import torch

import cache_reference as R
from gpu_helpers import to_f64

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _smla():
    from sparse_mla_attention_gb300 import build
    build.build()
    import sparse_mla_attention_gb300 as smla
    return smla


def _i32(x):
    return torch.as_tensor(np.ascontiguousarray(x, dtype=np.int32)).to(DEV)


class Pool:
    """Host copy (codes, scales, refcount) of a pool and the device handle on the same bytes."""

    def __init__(self, num_pages, page, block, seed=0, junk=True):
        rng = np.random.default_rng(seed)
        self.page, self.block, self.num_pages = page, block, num_pages
        self.codes = rng.integers(0, 256, size=(num_pages, page, 512), dtype=np.uint8)
        if junk:                                        # NaN codes wherever nothing is written later
            self.codes[rng.random((num_pages, page)) < 0.5] = 0x7F
        self.scales = np.exp2(rng.integers(-8, 3, size=(num_pages, page // block))).astype(np.float32)
        self.refcount = np.zeros(num_pages, dtype=np.int32)

    def device(self):
        smla = _smla()
        return smla.PagedCache(torch.from_numpy(self.codes.copy()).to(DEV).view(torch.float8_e4m3fn),
                               torch.from_numpy(self.scales.copy()).to(DEV),
                               torch.from_numpy(self.refcount.copy()).to(DEV))

    def check(self, cache, counts=True):
        got = cache.pages.view(torch.uint8).cpu().numpy()
        np.testing.assert_array_equal(got, self.codes)
        np.testing.assert_array_equal(cache.scales.cpu().numpy(), self.scales)
        if counts:
            np.testing.assert_array_equal(cache.refcount.cpu().numpy(), self.refcount)

    def place(self, lens, extra=1, seed=1):
        """Random pages for sequences of these lengths; returns the table."""
        rng = np.random.default_rng(seed)
        used = [-(-int(n) // self.page) for n in lens]
        table = np.full((len(lens), max(used + [0]) + extra), -1, dtype=np.int32)
        order = rng.permutation(self.num_pages)
        k = 0
        for b, n in enumerate(used):
            table[b, :n] = order[k:k + n]
            k += n
        assert k <= self.num_pages
        self.refcount[order[:k]] = 1
        return table

    def fill(self, table, lens, seed=2, amp=1.0):
        """Writes N(0, amp) rows as every sequence's content, through the host model."""
        rng = np.random.default_rng(seed)
        cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
        rows = bf16(rng.standard_normal((int(cu[-1]), 512)) * amp)
        R.write(self.codes, self.scales, table, np.zeros(len(lens), dtype=int), cu, rows, self.page, self.block)


def bf16(x):
    return torch.from_numpy(np.asarray(x, dtype=np.float32)).to(torch.bfloat16).double().numpy()


def bf16_dev(x):
    return torch.from_numpy(np.asarray(x, dtype=np.float32)).to(torch.bfloat16).to(DEV)


# ------------------------------------------------------------------------------------------------ writing rows
@pytest.mark.parametrize("page,block", [(16, 16), (64, 16), (64, 32), (64, 64), (256, 64)])
def test_write_matches_the_model(page, block):
    smla = _smla()
    rng = np.random.default_rng(page + block)
    starts = np.array([0, 5, block - 1, block, 3 * block + 7, page, 0, 2 * page + 1])
    counts = np.array([1, 1, 2, block, 2 * block + 3, page + 1, 3 * page, 0])
    pool = Pool(80, page, block, seed=3)
    table = pool.place(starts + counts)
    pool.fill(table, starts, seed=4)
    cu = np.concatenate([[0], np.cumsum(counts)])
    loud = np.exp2(rng.integers(-3, 4, size=(cu[-1], 1)))          # some scales grow, some do not
    rows = bf16(rng.standard_normal((cu[-1], 512)) * loud)
    cache = pool.device()
    smla.cache_write(cache, _i32(table), _i32(starts), _i32(cu), bf16_dev(rows))
    R.write(pool.codes, pool.scales, table, starts, cu, rows, page, block)
    pool.check(cache)
    # the same rows again at the same places: nothing changes
    smla.cache_write(cache, _i32(table), _i32(starts), _i32(cu), bf16_dev(rows))
    pool.check(cache)


def test_write_of_odd_values():
    smla = _smla()
    pool = Pool(12, 16, 16, seed=5)
    table = pool.place([16] * 10)
    rows = np.zeros((10, 512))
    rows[1, 3] = np.inf
    rows[1, 4] = -2.0
    rows[2, 5] = np.nan
    rows[2, 6] = 448.0
    rows[3, :] = np.inf                    # no finite value: the least scale
    rows[4, 0] = bf16(3.38e38)             # near the largest bf16
    rows[4, 1] = -1.0
    rows[5, :4] = [2.0 ** -126, -2.0 ** -130, 1e-38, 2.0 ** -133]      # bf16 subnormals under the least scale
    rows[6, :3] = [449.0, 450.0, -448.0]
    rows[7, :3] = [1.0, 2.0 ** -15, 3 * 2.0 ** -17]     # codes in e4m3's subnormal range, ties
    rows[8, :2] = [-0.0, 1.0]
    rows = bf16(rows)
    cu, start = np.arange(11), np.zeros(10, dtype=int)
    cache = pool.device()
    smla.cache_write(cache, _i32(table), _i32(start), _i32(cu), bf16_dev(rows))
    R.write(pool.codes, pool.scales, table, start, cu, rows, 16, 16)
    pool.check(cache)


def test_write_after_an_all_zero_block_and_token_by_token():
    smla = _smla()
    pool = Pool(6, 64, 32, seed=6)
    table = pool.place([100])
    cache = pool.device()
    rng = np.random.default_rng(7)
    tt = _i32(table)
    ws = smla.Workspace(DEV)
    for pos in range(70):
        row = bf16(rng.standard_normal((1, 512)) * (0.0 if pos < 3 else 2.0 ** (pos % 7)))
        cu, start = np.array([0, 1]), np.array([pos])
        smla.cache_write(cache, tt, _i32(start), _i32(cu), bf16_dev(row), workspace=ws)
        R.write(pool.codes, pool.scales, table, start, cu, row, 64, 32)
    pool.check(cache)


def test_write_bad_places_are_dropped_and_reported():
    smla = _smla()
    from sparse_mla_attention_gb300 import SmlaError, _lib
    pool = Pool(8, 16, 16, seed=8)
    table = pool.place([20, 16, 16, 16])
    bad = table.copy()
    bad[1, 0] = 8                           # past the pool
    bad[2, 0] = -1                          # no page
    start = np.array([16, 0, 0, 33])        # sequence 3 starts behind the table's last column
    cu = np.array([0, 2, 4, 6, 8])
    rows = bf16(np.random.default_rng(9).standard_normal((8, 512)))
    cache = pool.device()
    with pytest.raises(SmlaError) as e:
        smla.cache_write(cache, _i32(bad), _i32(start), _i32(cu), bf16_dev(rows))
    assert e.value.code == _lib.SMLA_ERR_INDEX
    R.write(pool.codes, pool.scales, table[:1], start[:1], cu[:2], rows[:2], 16, 16)
    pool.check(cache)
    # offsets that leave the rows or fall: dropped
    for cu in ([0, 2, 1, 3, 4], [0, 2, 4, 6, 90], [-3, 2, 4, 6, 8]):
        before = cache.pages.view(torch.uint8).clone()
        with pytest.raises(SmlaError) as e:
            smla.cache_write(cache, _i32(table), _i32(np.array([16, 40, 40, 40])), _i32(cu), bf16_dev(rows))
        assert e.value.code == _lib.SMLA_ERR_INDEX
        changed = (cache.pages.view(torch.uint8) != before).flatten(1).any(1).nonzero().flatten().tolist()
        assert set(changed) <= {int(table[0, 1])}


# ------------------------------------------------------------------------------------------------ pages
@pytest.mark.parametrize("num_pages,page", [(40, 64), (5000, 16), (70001, 16)])
def test_alloc_fork_free_compact_match_the_model(num_pages, page):
    smla = _smla()
    rng = np.random.default_rng(num_pages)
    block = 16
    pool = Pool(num_pages, page, block, seed=10)
    B = min(30, num_pages // 8)
    lens = rng.integers(0, 4 * page, size=B)
    lens[0] = 0
    table = np.full((B, 7), -1, dtype=np.int32)
    pool.refcount[rng.random(num_pages) < 0.4] = 3               # pages that others hold
    cache = pool.device()
    tt, ll = _i32(table), _i32(lens)

    smla.cache_alloc(cache, tt, ll)
    assert R.alloc(pool.refcount, table, lens, page)
    np.testing.assert_array_equal(tt.cpu().numpy(), table)
    lens = np.minimum(lens + rng.integers(0, page, size=B), 7 * page)   # they grow: only the missing pages come
    if R.alloc(pool.refcount, table, lens, page):
        ll = _i32(lens)
        smla.cache_alloc(cache, tt, ll)
        np.testing.assert_array_equal(tt.cpu().numpy(), table)
    pool.check(cache)

    parents = rng.integers(0, B, size=min(20, num_pages // 10))
    child = smla.cache_fork(cache, tt, ll, _i32(parents))
    want = R.fork(pool.codes, pool.scales, pool.refcount, table, lens, parents, page)
    np.testing.assert_array_equal(child.cpu().numpy(), want)
    pool.check(cache)

    rows = np.array([1, 0, len(parents) - 1])
    smla.cache_free(cache, child, _i32(rows))
    R.free_rows(pool.refcount, want, rows)
    smla.cache_free(cache, child, _i32(rows))                    # given back already: nothing to give
    np.testing.assert_array_equal(child.cpu().numpy(), want)
    pool.check(cache)

    both = torch.cat([tt, child])
    old = both.clone()
    new, count = smla.cache_compact(cache, both)
    model = np.concatenate([table, want])
    want_t, want_c = R.compact(pool.codes, pool.scales, pool.refcount, model)
    np.testing.assert_array_equal(new.cpu().numpy(), want_t)
    np.testing.assert_array_equal(count.cpu().numpy(), want_c)
    assert torch.equal(both, old)
    pool.check(cache)                                            # counts of the old pool are left
    # a compact pool stays as it is
    cache.refcount.copy_(count)
    again, count2 = smla.cache_compact(cache, new)
    assert torch.equal(again, new) and torch.equal(count2, count)
    smla.cache_free(cache, new)
    R.free_rows(want_c, want_t, range(len(want_t)))
    np.testing.assert_array_equal(cache.refcount.cpu().numpy(), want_c)


def test_too_few_pages_changes_nothing():
    smla = _smla()
    from sparse_mla_attention_gb300 import SmlaError, _lib
    pool = Pool(10, 16, 16, seed=11)
    lens = np.array([33, 30])
    table = pool.place(lens, extra=6)                            # 5 of 10 pages
    cache = pool.device()
    tt = _i32(table)
    with pytest.raises(SmlaError) as e:
        smla.cache_alloc(cache, tt, _i32([33 + 48, 30 + 48]))    # 6 more
    assert e.value.code == _lib.SMLA_ERR_PAGES
    np.testing.assert_array_equal(tt.cpu().numpy(), table)
    pool.check(cache)
    with pytest.raises(SmlaError) as e:
        smla.cache_fork(cache, tt, _i32(lens), _i32([0, 1, 0, 1, 0, 1]), out=(child := _i32(np.zeros((6, 9)))))
    assert e.value.code == _lib.SMLA_ERR_PAGES
    assert (child == -1).all()
    pool.check(cache)
    smla.cache_alloc(cache, tt, _i32([33 + 32, 30 + 48]))        # exactly the 5 that are left
    assert R.alloc(pool.refcount, table, [65, 78], 16)
    np.testing.assert_array_equal(tt.cpu().numpy(), table)
    pool.check(cache)


def test_bad_page_calls_are_reported():
    smla = _smla()
    from sparse_mla_attention_gb300 import SmlaError, _lib
    pool = Pool(10, 16, 16, seed=12)
    lens = np.array([33, 20])
    table = pool.place(lens)
    cache = pool.device()

    def code(f, *a, **k):
        with pytest.raises(SmlaError) as e:
            f(*a, **k)
        return e.value.code
    bad = _i32(np.zeros((2, 4)))
    assert code(smla.cache_fork, cache, _i32(table), _i32(lens), _i32([2, -1]), out=bad) == _lib.SMLA_ERR_INDEX
    assert (bad == -1).all()
    pool.check(cache)
    # a table that names pages out of the pool
    wild = table.copy()
    wild[0, 0], wild[1, 1] = 10, -7
    child = _i32(np.zeros((2, 4)))
    assert code(smla.cache_fork, cache, _i32(wild), _i32(lens), _i32([0, 1]), out=child) == _lib.SMLA_ERR_INDEX
    assert child[0, 0] == -1 and child[0, 1] == int(table[0, 1]) and child[1, 1] == -1
    new = int(child[0, 2])
    assert new == np.nonzero(pool.refcount == 0)[0][0]
    pool.codes[new], pool.scales[new] = pool.codes[table[0, 2]], pool.scales[table[0, 2]]
    smla.cache_free(cache, child)
    pool.check(cache)
    # giving back a page that nobody holds
    empty = np.full((1, 4), -1)
    empty[0, 2] = int(np.nonzero(pool.refcount == 0)[0][0])
    t = _i32(empty)
    assert code(smla.cache_free, cache, t) == _lib.SMLA_ERR_REFCOUNT
    assert (t == -1).all()
    assert code(smla.cache_free, cache, _i32(table), _i32([5])) == _lib.SMLA_ERR_INDEX
    pool.check(cache)
    # a row listed twice is given back once
    t = _i32(table)
    smla.cache_free(cache, t, _i32([1, 1]))
    R.free_rows(pool.refcount, table, [1])
    pool.check(cache)


def test_copy_pages():
    smla = _smla()
    from sparse_mla_attention_gb300 import SmlaError, _lib
    for page, block in ((16, 16), (128, 32), (256, 64)):
        pool = Pool(50, page, block, seed=13)
        cache = pool.device()
        src, dst = np.array([3, 3, 49, 7, 0]), np.array([10, 11, 1, 40, 48])
        smla.cache_copy_pages(cache, _i32(src), _i32(dst))
        pool.codes[dst], pool.scales[dst] = pool.codes[src], pool.scales[src]
        pool.check(cache)
        for s, d in (([1, 2], [5, 5]), ([1, 5], [5, 6]), ([4], [4])):
            with pytest.raises(SmlaError) as e:
                smla.cache_copy_pages(cache, _i32(s), _i32(d))
            assert e.value.code == _lib.SMLA_ERR_OVERLAP
            pool.check(cache)
        with pytest.raises(SmlaError) as e:
            smla.cache_copy_pages(cache, _i32([50, 2, -1]), _i32([6, 8, 9]))
        assert e.value.code == _lib.SMLA_ERR_INDEX
        pool.codes[8], pool.scales[8] = pool.codes[2], pool.scales[2]
        pool.check(cache)
        smla.cache_copy_pages(cache, _i32([]), _i32([]))


# ------------------------------------------------------------------------------------------------ attention
def _attend_and_check(pool, table, lens, H, seed, topk=None, seq=None, sink=True, scale=None, q=None):
    smla = _smla()
    rng = np.random.default_rng(seed)
    T = len(lens)
    q = bf16(rng.standard_normal((T, H, 512)) if q is None else q)
    sk = rng.standard_normal(H).astype(np.float32) if sink else None
    cache = pool.device()
    o, lse = smla.sparse_mla_fwd_paged(
        bf16_dev(q), cache, _i32(table), _i32(lens), topk=None if topk is None else _i32(topk),
        seq=None if seq is None else _i32(seq), sink=None if sk is None else torch.from_numpy(sk).to(DEV),
        scale=scale)
    ref, rl, ob, lb = R.attend(q, pool.codes, pool.scales, table, lens, pool.page, pool.block, topk, seq,
                               None if sk is None else sk.astype(np.float64), scale)
    got, gl = to_f64(o), lse.double().cpu().numpy()
    assert np.isfinite(got).all()
    over = np.abs(got - ref) - ob
    assert over.max() <= 0, f"o off by {over.max():.3e} over its bound at {np.unravel_index(over.argmax(), over.shape)}"
    none = np.isneginf(rl)
    np.testing.assert_array_equal(np.isneginf(gl), none)
    over = np.abs(gl - rl)[~none] - lb[~none]
    assert over.size == 0 or over.max() <= 0, f"lse off by {over.max():.3e} over its bound"
    pool.check(cache)
    return o, lse


LENS = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 333]


@pytest.mark.parametrize("H", [16, 32, 48, 64, 80, 96, 112, 128])
@pytest.mark.parametrize("page,block", [(16, 16), (64, 32), (256, 64)])
def test_attention_over_all_positions(H, page, block):
    pool = Pool(80, page, block, seed=20)
    table = pool.place(LENS)
    pool.fill(table, LENS)
    _attend_and_check(pool, table, LENS, H, seed=H, sink=H % 32 == 0)


@pytest.mark.parametrize("H,K", [(16, 1), (16, 70), (64, 64), (64, 300), (96, 17), (128, 512), (128, 513), (112, 129)])
def test_attention_over_picks(H, K):
    rng = np.random.default_rng(K)
    pool = Pool(60, 64, 32, seed=21)
    lens = [700, 1, 0, 64, 333, 900]
    table = pool.place(lens)
    pool.fill(table, lens)
    topk = np.full((len(lens), K), -1, dtype=np.int32)
    for t, n in enumerate(lens):
        if n:
            topk[t] = rng.integers(0, n, size=K)
            topk[t, rng.random(K) < 0.3] = -1
    topk[3] = -1                                       # a token whose mask leaves nothing
    topk[4, K // 2:] = -1
    if K > 2:
        topk[5, 1] = topk[5, 0] = 899                  # the same position twice
    _attend_and_check(pool, table, lens, H, seed=K, topk=topk, sink=K % 2 == 0)


@pytest.mark.parametrize("H,new,K", [(16, 4, 0), (64, 2, 0), (128, 3, 0), (32, 5, 40)])
def test_several_tokens_of_a_sequence(H, new, K):
    rng = np.random.default_rng(H)
    pool = Pool(60, 32, 16, seed=22)
    total = [200, 7, 64, 129]
    table = pool.place(total)
    pool.fill(table, total)
    seq = np.repeat(np.arange(4), new)[::-1].copy()    # in any order
    lens = np.array([max(0, total[b] - i % new) for i, b in enumerate(seq)])
    lens[2] = 0                                        # a padded slot
    topk = None
    if K:
        topk = np.array([rng.integers(-1, max(n, 1), size=K) if n else np.full(K, -1) for n in lens])
    _attend_and_check(pool, table, lens, H, seed=H, topk=topk, seq=seq)


@pytest.mark.parametrize("H", [16, 64, 128])
def test_long_sequences_are_split(H):
    lens = [20011, 3, 4097]
    pool = Pool(400, 64, 64, seed=23)
    table = pool.place(lens)
    pool.fill(table, lens)
    _attend_and_check(pool, table, lens, H, seed=H)


@pytest.mark.parametrize("H,page", [(128, 64), (64, 16)])
def test_many_tiles_and_sequences_for_each_processor(H, page):
    # tens of tiles and several items for each of the GPU's SMs: every buffer and barrier comes round
    rng = np.random.default_rng(H)
    lens = [9000, 1, 64, 5000, 700, 700, 65, 4000, 0, 0, 3] + [int(n) for n in rng.integers(1, 2500, size=33)]
    lens = lens if H == 128 else [2 * n for n in lens]
    pool = Pool(sum(-(-n // page) for n in lens) + 2, page, 16, seed=33)
    table = pool.place(lens)
    pool.fill(table, lens)
    _attend_and_check(pool, table, lens, H, seed=34)


@pytest.mark.parametrize("H,T", [(128, 300), (48, 700)])
def test_many_tokens_with_picks(H, T):
    rng = np.random.default_rng(T)
    lens_b = [3000, 700, 5000]
    pool = Pool(150, 64, 32, seed=35)
    table = pool.place(lens_b)
    pool.fill(table, lens_b)
    seq = rng.integers(0, 3, size=T)
    lens = np.array([rng.integers(1, lens_b[b] + 1) for b in seq])
    K = 449
    topk = np.array([rng.integers(0, n, size=K) for n in lens])
    # whole tiles without a valid rank, in front, behind, and everywhere
    for t in range(0, T, 7):
        topk[t, :64 * (t % 8)] = -1
    for t in range(3, T, 11):
        topk[t, 64 * (t % 7):] = -1
    _attend_and_check(pool, table, lens, H, seed=36, topk=topk, seq=seq, sink=H == 48)


def test_scales_of_every_size_and_scores_far_apart():
    # rows whose blocks' scales differ by 2^20, scores that rise along the sequence
    # (the running maximum grows again and again), and one row that outweighs all others
    pool = Pool(60, 64, 16, seed=24, junk=False)
    lens = [1000, 500]
    table = pool.place(lens)
    rng = np.random.default_rng(25)
    cu = np.array([0, 1000, 1500])
    amp = np.concatenate([np.exp2(-20 + 20 * np.arange(1000) / 1000), np.full(500, 0.05)])
    rows = rng.standard_normal((1500, 512)) * amp[:, None]
    rows[1100] = 1.0
    R.write(pool.codes, pool.scales, table, [0, 0], cu, bf16(rows), 64, 16)
    q = rng.standard_normal((2, 64, 512))
    q[:, ::2] += 1.0                                   # heads drawn to row 1100 and to loud rows
    _attend_and_check(pool, table, lens, 64, seed=26, q=q)
    _attend_and_check(pool, table, lens, 64, seed=26, q=q * 8, sink=False)


def test_one_position_gives_its_row():
    # a single rank without a sink has weight 1: o is the cache row rounded to bf16 (exact: 4 significant bits)
    smla = _smla()
    pool = Pool(10, 16, 16, seed=27)
    lens = [1, 33]
    table = pool.place(lens)
    pool.fill(table, lens)
    topk = np.array([[0, -1, -1], [-1, 32, -1]])
    o, _ = _attend_and_check(pool, table, lens, 16, seed=28, topk=topk, sink=False)
    for t, p in ((0, 0), (1, 32)):
        x, _, _ = R.rows_of(pool.codes, pool.scales, table[t], np.array([p]), 16, 16)
        np.testing.assert_array_equal(to_f64(o)[t], np.broadcast_to(x, (16, 512)))


def test_nan_and_inf_reach_only_those_who_see_them():
    smla = _smla()
    pool = Pool(20, 16, 16, seed=29, junk=False)
    lens = [40, 40, 25]
    table = pool.place(lens)
    pool.fill(table, lens)
    pool.codes[table[0, 2], 3] = 0x7F                  # position 35 of sequence 0
    cache = pool.device()
    q = bf16_dev(np.random.default_rng(30).standard_normal((3, 32, 512)))
    o, lse = smla.sparse_mla_fwd_paged(q, cache, _i32(table), _i32(lens))
    assert o[0].isnan().all() and lse[0].isnan().all()
    assert o[1:].isfinite().all() and lse[1:].isfinite().all()
    o, lse = smla.sparse_mla_fwd_paged(q, cache, _i32(table), _i32([35, 40, 25]))
    assert o.isfinite().all() and lse.isfinite().all()
    q[1, 5, 7] = float("inf")
    o, lse = smla.sparse_mla_fwd_paged(q, cache, _i32(table), _i32([35, 40, 25]))
    bad = (~o.isfinite()).any(2)
    assert bad[1, 5] and bad.sum() == 1


def test_bad_indices_are_masked_and_reported():
    smla = _smla()
    from sparse_mla_attention_gb300 import SmlaError, _lib
    pool = Pool(20, 16, 16, seed=31)
    lens = [40, 30]
    table = pool.place(lens)
    pool.fill(table, lens)
    cache = pool.device()
    q = bf16(np.random.default_rng(32).standard_normal((2, 16, 512)))

    def run(tab, ln, topk=None, seq=None):
        out = (torch.zeros((2, 16, 512), dtype=torch.bfloat16, device=DEV), torch.zeros((2, 16), device=DEV))
        with pytest.raises(SmlaError) as e:
            smla.sparse_mla_fwd_paged(bf16_dev(q), cache, _i32(tab), _i32(ln), topk=None if topk is None else _i32(topk),
                                      seq=None if seq is None else _i32(seq), out=out)
        assert e.value.code == _lib.SMLA_ERR_INDEX
        return out

    def same(out, ln, topk=None, rows=(0, 1)):
        ref, rl, ob, lb = R.attend(q, pool.codes, pool.scales, table, ln, 16, 16, topk)
        for t in rows:
            assert (np.abs(to_f64(out[0])[t] - ref[t]) <= ob[t]).all()
            assert ((np.abs(out[1].double().cpu().numpy()[t] - rl[t]) <= lb[t]) | np.isneginf(rl[t])).all()
    wild = table.copy()
    wild[0, 1] = 20                                    # positions 16..31 of sequence 0 have no page
    topk = np.stack([np.concatenate([np.arange(16), np.arange(32, 40)])] * 2)
    ref, rl, ob, lb = R.attend(q[:1], pool.codes, pool.scales, table, [40], 16, 16, topk[:1])
    out = run(wild, lens)
    assert (np.abs(to_f64(out[0])[0] - ref[0]) <= ob[0]).all()
    # picks past the length, and below -1
    picks = np.array([[3, 40, -2, 7], [30, 5, 1 << 30, -(1 << 31)]], dtype=np.int64).astype(np.int32)
    out = run(table, lens, topk=picks)
    same(out, lens, topk=np.array([[3, -1, -1, 7], [-1, 5, -1, -1]]))
    # a length past the table, and a negative one
    out = run(table, [16 * table.shape[1] + 1, -5])
    assert (out[0][1] == 0).all() and torch.isneginf(out[1][1]).all()
    # a sequence that is not there
    out = run(table, lens, seq=[0, 2])
    same(out, lens, rows=(0,))
    assert (out[0][1] == 0).all()
    out = run(table, lens, seq=[-1, 1])
    same(out, lens, rows=(1,))


# ------------------------------------------------------------------------------------------------ together
def test_serving_run():
    """Allocate, write prompts, answer, fork, go on token by token, give back and compact, the
    attention checked after each stage; a stream other than the default one; workspaces kept."""
    smla = _smla()
    page, block, H = 32, 16, 48
    rng = np.random.default_rng(40)
    pool = Pool(64, page, block, seed=41)
    cache = pool.device()
    ws = smla.Workspace(DEV)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        lens = np.array([45, 64, 1])
        table = np.full((3, 6), -1, dtype=np.int32)
        tt = _i32(table)

        def attend(tt, table, lens):
            q = bf16(rng.standard_normal((len(lens), H, 512)))
            o, lse = smla.sparse_mla_fwd_paged(bf16_dev(q), cache, tt, _i32(lens), workspace=ws)
            ref, rl, ob, lb = R.attend(q, pool.codes, pool.scales, table, lens, page, block)
            assert (np.abs(to_f64(o) - ref) <= ob).all()
            assert (np.abs(lse.double().cpu().numpy() - rl) <= lb).all()

        def grow(tt, table, lens, counts):
            new = lens + counts
            smla.cache_alloc(cache, tt, _i32(new), workspace=ws)
            assert R.alloc(pool.refcount, table, new, page)
            cu = np.concatenate([[0], np.cumsum(counts)])
            rows = bf16(rng.standard_normal((cu[-1], 512)) * 2)
            smla.cache_write(cache, tt, _i32(lens), _i32(cu), bf16_dev(rows), workspace=ws)
            R.write(pool.codes, pool.scales, table, lens, cu, rows, page, block)
            attend(tt, table, new)
            return new
        lens = grow(tt, table, np.zeros(3, dtype=int), lens)
        parents = np.array([0, 1, 1, 0])
        child = smla.cache_fork(cache, tt, _i32(lens), _i32(parents), workspace=ws)
        table = np.concatenate([table, R.fork(pool.codes, pool.scales, pool.refcount, table, lens, parents, page)])
        tt = torch.cat([tt, child])
        lens = np.concatenate([lens, lens[parents]])
        for step in range(4):
            lens = grow(tt, table, lens, np.ones(7, dtype=int))
        smla.cache_free(cache, tt, _i32([0, 4]), workspace=ws)
        R.free_rows(pool.refcount, table, [0, 4])
        lens[[0, 4]] = 0
        tt, count = smla.cache_compact(cache, tt, workspace=ws)
        cache.refcount.copy_(count)
        table, pool.refcount = R.compact(pool.codes, pool.scales, pool.refcount, table)
        np.testing.assert_array_equal(tt.cpu().numpy(), table)
        keep = np.array([1, 2, 3, 5, 6])
        tt, table, lens = tt[keep.tolist()].contiguous(), table[keep], lens[keep]
        lens = grow(tt, table, lens, np.array([1, 40, 1, 3, 1]))
        # written places alone are compared: pages given back keep old bytes in both
        pool.check(cache)
    torch.cuda.current_stream().wait_stream(side)


def test_a_captured_step_replays():
    """One decode step (alloc, write, attend, fork, free) captured into a graph and replayed with
    new lengths, rows and queries; two graphs on one workspace, in turn."""
    smla = _smla()
    page, block, H, B = 16, 16, 64, 3
    rng = np.random.default_rng(50)
    pool = Pool(40, page, block, seed=51)
    cache = pool.device()
    lens = np.array([15, 30, 3])
    table = np.full((B, 5), -1, dtype=np.int32)
    tt, start, end = _i32(table), _i32(np.zeros(B)), _i32(lens)
    smla.cache_alloc(cache, tt, end)
    assert R.alloc(pool.refcount, table, lens, page)
    cu = np.concatenate([[0], np.cumsum(lens)])
    rows = bf16(rng.standard_normal((cu[-1], 512)))
    smla.cache_write(cache, tt, start, _i32(cu), bf16_dev(rows))
    R.write(pool.codes, pool.scales, table, np.zeros(B, dtype=int), cu, rows, page, block)

    one, row_t, q_t = _i32(np.arange(B + 1)), bf16_dev(np.zeros((B, 512))), bf16_dev(np.zeros((B, H, 512)))
    parents = _i32([2, 0])
    child = _i32(np.full((2, 5), -1))
    o, lse = torch.empty((B, H, 512), dtype=torch.bfloat16, device=DEV), torch.empty((B, H), device=DEV)
    ws = smla.Workspace(DEV)
    ws.get(64 << 20)
    kw = dict(workspace=ws, check_status=False)

    def step():
        smla.cache_free(cache, child, **kw)
        smla.cache_alloc(cache, tt, end, **kw)
        smla.cache_write(cache, tt, start, one, row_t, **kw)
        smla.sparse_mla_fwd_paged(q_t, cache, tt, end, out=(o, lse), **kw)
        smla.cache_fork(cache, tt, end, parents, out=child, **kw)

    def attend_only():
        smla.sparse_mla_fwd_paged(q_t, cache, tt, end, out=(o, lse), **kw)
    graphs = []
    for f in (step, attend_only):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f()
        graphs.append(g)
    kids = np.full((2, 5), -1, dtype=np.int32)
    for i in range(6):
        new = lens + 1
        row = bf16(rng.standard_normal((B, 512)) * (i + 1))
        q = bf16(rng.standard_normal((B, H, 512)))
        start.copy_(_i32(lens)); end.copy_(_i32(new)); row_t.copy_(bf16_dev(row)); q_t.copy_(bf16_dev(q))
        graphs[0].replay()
        R.free_rows(pool.refcount, kids, range(2))
        assert R.alloc(pool.refcount, table, new, page)
        R.write(pool.codes, pool.scales, table, lens, np.arange(B + 1), row, page, block)
        ref, rl, ob, lb = R.attend(q, pool.codes, pool.scales, table, new, page, block)
        kids = R.fork(pool.codes, pool.scales, pool.refcount, table, new, [2, 0], page)
        assert (np.abs(to_f64(o) - ref) <= ob).all()
        np.testing.assert_array_equal(tt.cpu().numpy(), table)
        np.testing.assert_array_equal(child.cpu().numpy(), kids)
        pool.check(cache)
        first = o.clone()
        o.zero_(); lse.zero_()
        graphs[1].replay()
        assert torch.equal(o, first)                   # the same call gives the same bits
        assert (np.abs(lse.double().cpu().numpy() - rl) <= lb).all()
        lens = new


def test_results_do_not_depend_on_the_run():
    pool = Pool(400, 64, 32, seed=60)
    lens = [9001, 4000, 77]
    table = pool.place(lens)
    pool.fill(table, lens)
    smla = _smla()
    cache = pool.device()
    q = bf16_dev(np.random.default_rng(61).standard_normal((3, 128, 512)))
    runs = [smla.sparse_mla_fwd_paged(q, cache, _i32(table), _i32(lens)) for _ in range(3)]
    for o, lse in runs[1:]:
        assert torch.equal(o, runs[0][0]) and torch.equal(lse, runs[0][1])


def test_pages_past_four_gigabytes():
    # a pool of 4.5 GB: rows behind byte offset 2^32
    smla = _smla()
    page, n = 256, 36000
    cache = smla.PagedCache.empty(n, page, 64)
    table = np.array([[n - 1, 5, n - 2]], dtype=np.int32)
    rows = bf16(np.random.default_rng(70).standard_normal((600, 512)))
    smla.cache_write(cache, _i32(table), _i32([0]), _i32([0, 600]), bf16_dev(rows))
    cache.refcount[[n - 1, 5, n - 2]] = 1
    small = Pool(3, page, 64, seed=71)
    R.write(small.codes, small.scales, np.array([[0, 1, 2]]), [0], [0, 600], rows, page, 64)
    at = [n - 1, 5, n - 2]
    got = cache.pages.view(torch.uint8)[at].cpu().numpy().reshape(-1, 512)[:600]
    np.testing.assert_array_equal(got, small.codes.reshape(-1, 512)[:600])
    q = bf16(np.random.default_rng(72).standard_normal((1, 64, 512)))
    o, lse = smla.sparse_mla_fwd_paged(bf16_dev(q), cache, _i32(table), _i32([600]))
    ref, rl, ob, lb = R.attend(q, small.codes, small.scales, np.array([[0, 1, 2]]), [600], page, 64)
    assert (np.abs(to_f64(o) - ref) <= ob).all()
    new, _ = smla.cache_compact(cache, _i32(table))
    np.testing.assert_array_equal(new.cpu().numpy(), [[2, 0, 1]])      # page 5 moves too: three live pages
    o2, lse2 = smla.sparse_mla_fwd_paged(bf16_dev(q), cache, new, _i32([600]))
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
