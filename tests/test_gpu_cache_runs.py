"""GPU tests of the paged 8-bit cache at sizes that keep every processor at work for
several turns, of calls that run at once, and of what a call must leave alone.

Models, bounds and the pool are those of test_gpu_cache.
"""

import numpy as np
import pytest
import torch

import cache_reference as R
from gpu_helpers import to_f64
from test_gpu_cache import DEV, Pool, _attend_and_check, _i32, _smla, bf16, bf16_dev

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------------------ writing rows
@pytest.mark.parametrize("page,block", [(16, 16), (128, 32), (64, 64)])
def test_long_ragged_prompts(page, block):
    # more blocks than CTAs: 1216 of 16 rows, 608 of 32 or 304 of 64 are worked on at a time
    smla = _smla()
    rng = np.random.default_rng(block)
    B = 36
    counts = rng.integers(1, 2 * 32000 // B, size=B)
    counts[[3, 20]] = 0
    starts = rng.integers(0, 300, size=B)
    starts[::5] = 0
    pool = Pool(int((-(-(starts + counts) // page)).sum()) + 5, page, block, seed=block, junk=False)
    table = pool.place(starts + counts)
    pool.fill(table, starts, seed=4)
    cu = np.concatenate([[0], np.cumsum(counts)])
    rows = bf16(rng.standard_normal((cu[-1] + 3, 512)) * np.exp2(rng.integers(-3, 4, size=(cu[-1] + 3, 1))))
    cache = pool.device()
    smla.cache_write(cache, _i32(table), _i32(starts), _i32(cu), bf16_dev(rows))      # three rows nobody names
    R.write(pool.codes, pool.scales, table, starts, cu, rows, page, block)
    pool.check(cache)


def test_one_bad_place_in_a_long_write():
    # a missing page in the middle: its rows are dropped and reported, all others are written
    smla = _smla()
    from sparse_mla_attention_gb300 import SmlaError, _lib
    page = block = 16
    counts = np.array([9000, 7000, 12000])
    pool = Pool(1800, page, block, seed=5, junk=False)
    table = pool.place(counts)
    cu = np.concatenate([[0], np.cumsum(counts)])
    rows = bf16(np.random.default_rng(6).standard_normal((cu[-1], 512)))
    bad = table.copy()
    bad[1, 200] = -1
    cache = pool.device()
    with pytest.raises(SmlaError) as e:
        smla.cache_write(cache, _i32(bad), _i32([0, 0, 0]), _i32(cu), bf16_dev(rows))
    assert e.value.code == _lib.SMLA_ERR_INDEX
    kept = pool.codes[table[1, 200]].copy(), pool.scales[table[1, 200]].copy()
    R.write(pool.codes, pool.scales, table, [0, 0, 0], cu, rows, page, block)
    pool.codes[table[1, 200]], pool.scales[table[1, 200]] = kept
    pool.check(cache)
    # the word of a call is its own: a good call on the same workspace reports nothing
    ws = smla.Workspace(DEV)
    smla.cache_write(cache, _i32(bad), _i32([0, 0, 0]), _i32(cu), bf16_dev(rows), workspace=ws, check_status=False)
    smla.cache_write(cache, _i32(table), _i32([0, 0, 0]), _i32(cu), bf16_dev(rows), workspace=ws)
    R.write(pool.codes, pool.scales, table, [0, 0, 0], cu, rows, page, block)
    pool.check(cache)


# ------------------------------------------------------------------------------------------------ pages
@pytest.mark.parametrize("page,block,pairs", [(16, 16, 4500), (32, 16, 2100), (64, 64, 1100), (128, 64, 601),
                                              (256, 32, 300)])
def test_copies_of_many_pages(page, block, pairs):
    # more than six pieces for each of 152 CTAs, so that their slots come round
    smla = _smla()
    rng = np.random.default_rng(page)
    pool = Pool(2 * pairs + 3, page, block, seed=page, junk=False)
    order = rng.permutation(2 * pairs + 3)
    src, dst = order[:pairs], order[pairs:2 * pairs]
    src[1] = src[0]                                             # one page to two places
    cache = pool.device()
    smla.cache_copy_pages(cache, _i32(src), _i32(dst))
    pool.codes[dst], pool.scales[dst] = pool.codes[src], pool.scales[src]
    pool.check(cache)


@pytest.mark.parametrize("B,max_pages", [(40, 13), (900, 36), (901, 50)])
def test_frees_small_and_large(B, max_pages):
    # up to 32768 entries a cluster takes the call, above them the whole GPU
    smla = _smla()
    from sparse_mla_attention_gb300 import SmlaError, _lib
    rng = np.random.default_rng(B)
    num = B * max_pages // 2
    cache = smla.PagedCache(torch.empty((num, 16, 512), dtype=torch.float8_e4m3fn, device=DEV),
                            torch.zeros((num, 1), device=DEV), torch.zeros(num, dtype=torch.int32, device=DEV))
    table = rng.integers(-1, num, size=(B, max_pages)).astype(np.int32)
    count = np.bincount(table[table >= 0], minlength=num).astype(np.int32) + rng.integers(0, 2, size=num).astype(np.int32)
    cache.refcount.copy_(_i32(count))
    tt = _i32(table)
    rows = np.concatenate([np.arange(1, B), [1, 1]])            # row 0 stays, row 1 is listed three times
    smla.cache_free(cache, tt, _i32(rows))
    R.free_rows(count, table, range(1, B))
    np.testing.assert_array_equal(tt.cpu().numpy(), table)
    np.testing.assert_array_equal(cache.refcount.cpu().numpy(), count)
    # a number past the pool, a free page and a row past the table: reported, the rest given back
    want = count.copy()
    R.free_rows(want, table, [0])
    free = int(np.flatnonzero(want == 0)[0]) if (want == 0).any() else None
    table[:] = -1
    table[0] = tt[0].cpu().numpy()
    for row, entry, listed, code in ((1, num, 1, _lib.SMLA_ERR_INDEX), (2, free, 2, _lib.SMLA_ERR_REFCOUNT),
                                     (3, -1, B, _lib.SMLA_ERR_INDEX)):
        if entry is None:
            continue
        bad = table.copy()
        bad[row, max_pages - 1] = entry
        cache.refcount.copy_(_i32(count))
        tt = _i32(bad)
        rows = np.resize(np.array([0, listed]), B + 1)
        with pytest.raises(SmlaError) as e:
            smla.cache_free(cache, tt, _i32(rows))
        assert e.value.code == code
        np.testing.assert_array_equal(cache.refcount.cpu().numpy(), want)
        assert (tt.cpu().numpy()[:3] == -1).all()


def test_a_captured_compaction_replays():
    smla = _smla()
    page, block = 64, 16
    rng = np.random.default_rng(8)
    pool = Pool(700, page, block, seed=9, junk=False)
    cache = pool.device()
    tt, ll = _i32(np.full((50, 9), -1)), _i32(np.zeros(50))
    new, count = torch.empty_like(tt), torch.empty_like(cache.refcount)
    ws = smla.Workspace(DEV)
    ws.get(64 << 20)
    kw = dict(workspace=ws, check_status=False)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        smla.cache_alloc(cache, tt, ll, **kw)
        smla.cache_compact(cache, tt, out=(new, count), **kw)
    for i in range(4):
        pool.refcount[:] = 0
        table = np.full((50, 9), -1, dtype=np.int32)
        held = rng.random(700) < 0.3                            # pages that others hold
        pool.refcount[held] = 2
        lens = rng.integers(0, 9 * page // 2, size=50)
        cache.refcount.copy_(_i32(pool.refcount)); tt.fill_(-1); ll.copy_(_i32(lens))
        g.replay()
        assert R.alloc(pool.refcount, table, lens, page)
        np.testing.assert_array_equal(tt.cpu().numpy(), table)
        want, want_count = R.compact(pool.codes, pool.scales, pool.refcount, table)
        np.testing.assert_array_equal(new.cpu().numpy(), want)
        np.testing.assert_array_equal(count.cpu().numpy(), want_count)
        pool.check(cache)


# ------------------------------------------------------------------------------------------------ attention
def test_a_position_picked_twice_counts_twice():
    pool = Pool(20, 16, 16, seed=10)
    lens = [100, 40, 7]
    table = pool.place(lens)
    pool.fill(table, lens)
    rng = np.random.default_rng(11)
    topk = np.stack([rng.integers(0, n, size=150) for n in lens]).astype(np.int64)
    topk[1, :] = 39                                             # one row 150 times
    topk[2, 1::2] = -1
    _attend_and_check(pool, table, lens, 80, 12, topk=topk)


def test_many_short_tokens():
    # more tokens than threads that look for a CTA's first one; most see a row or none
    T = 1500
    rng = np.random.default_rng(13)
    lens = rng.integers(0, 4, size=T)
    lens[700] = 200
    pool = Pool(60, 16, 16, seed=14)
    table = pool.place([200] * 4)
    pool.fill(table, [200] * 4)
    _attend_and_check(pool, table, lens, 16, 15, seq=rng.integers(0, 4, size=T))


@pytest.mark.parametrize("H", [16, 80, 112])
def test_memory_behind_the_outputs_stays(H):
    smla = _smla()
    rng = np.random.default_rng(H)
    T, extra = 5, 3
    pool = Pool(200, 32, 32, seed=16)
    lens = [700, 0, 33, 64, 1200]
    table = pool.place(lens)
    pool.fill(table, lens)
    cache = pool.device()
    q = bf16(rng.standard_normal((T, H, 512)))
    o = torch.full((T + extra, H, 512), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((T + extra, H), 7.0, device=DEV)
    smla.sparse_mla_fwd_paged(bf16_dev(q), cache, _i32(table), _i32(lens), out=(o[:T], lse[:T]))
    assert (o[T:] == 7.0).all() and (lse[T:] == 7.0).all()
    ref, rl, ob, lb = R.attend(q, pool.codes, pool.scales, table, lens, 32, 32)
    assert (np.abs(to_f64(o[:T]) - ref) <= ob).all()
    pool.check(cache)


def test_calls_at_once_on_two_streams():
    # each stream has its workspace; both read one pool, and one of them writes pages of its own
    smla = _smla()
    rng = np.random.default_rng(17)
    page, block, H = 64, 32, 128
    pool = Pool(700, page, block, seed=18)
    lens = [9000, 300, 5000, 1, 0, 12000]
    table = pool.place(lens)
    pool.fill(table, lens)
    fresh = np.array([[p for p in range(700) if pool.refcount[p] == 0][:100]], dtype=np.int32)
    cache = pool.device()
    q = [bf16_dev(rng.standard_normal((6, H, 512))) for _ in range(2)]
    topk = _i32(np.where(np.array(lens)[:, None] > 0, rng.integers(0, np.maximum(lens, 1)[:, None], size=(6, 500)), -1))
    rows = bf16(rng.standard_normal((6000, 512)))
    tt, ll, ft, cu, start, rt = _i32(table), _i32(lens), _i32(fresh), _i32([0, 6000]), _i32([0]), bf16_dev(rows)
    alone = [smla.sparse_mla_fwd_paged(q[0], cache, tt, ll), smla.sparse_mla_fwd_paged(q[1], cache, tt, ll, topk=topk)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    work = [smla.Workspace(DEV), smla.Workspace(DEV)]
    got = [[], []]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for i in range(8):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                kw = dict(workspace=work[k], check_status=False)
                got[k].append(smla.sparse_mla_fwd_paged(q[k], cache, tt, ll, topk=topk if k else None, **kw))
                if k:
                    smla.cache_write(cache, ft, start, cu, rt, **kw)
    torch.cuda.synchronize()
    for k in range(2):
        for o, lse in got[k]:
            assert torch.equal(o, alone[k][0]) and torch.equal(lse, alone[k][1])
    R.write(pool.codes, pool.scales, fresh, [0], [0, 6000], rows, page, block)
    pool.check(cache)


@pytest.mark.parametrize("picks", [False, True])
def test_padded_slots_hold_anything(picks):
    # a captured step's batch is filled up with slots of length 0, whatever their other entries say
    smla = _smla()
    rng = np.random.default_rng(21)
    pool = Pool(40, 16, 16, seed=22)
    table = pool.place([100, 230])
    pool.fill(table, [100, 230])
    cache = pool.device()
    lens = np.array([100, 0, 230, 0, 0, 0])
    seq = np.array([0, -1, 1, 2, 1 << 30, -(1 << 31)], dtype=np.int64)
    topk = rng.integers(-(1 << 31), 1 << 31, size=(6, 70), dtype=np.int64)
    topk[0], topk[2] = rng.integers(0, 100, size=70), rng.integers(0, 230, size=70)
    q = bf16(rng.standard_normal((6, 32, 512)))
    sink = rng.standard_normal(32).astype(np.float32)
    o, lse = smla.sparse_mla_fwd_paged(bf16_dev(q), cache, _i32(table), _i32(lens), topk=_i32(topk) if picks else None,
                                       seq=_i32(seq), sink=torch.from_numpy(sink).to(DEV))
    live = [0, 2]
    ref, rl, ob, lb = R.attend(q[live], pool.codes, pool.scales, table, lens[live], 16, 16,
                               topk[live] if picks else None, None, sink.astype(np.float64))
    assert (np.abs(to_f64(o)[live] - ref) <= ob).all()
    assert (np.abs(lse.double().cpu().numpy()[live] - rl) <= lb).all()
    for t in (1, 3, 4, 5):
        assert (o[t] == 0).all()
        # log2(e) and back, and a sum of one: four roundings of 2^-24
        assert (np.abs(lse.double().cpu().numpy()[t] - sink) <= 2.0 ** -22 * np.abs(sink)).all()


def test_empty_batches():
    # a step in which no sequence is left: every call does nothing and reports nothing
    smla = _smla()
    pool = Pool(8, 16, 16, seed=20)
    cache = pool.device()
    ws = smla.Workspace(DEV)
    none, table = _i32([]), torch.empty((0, 3), dtype=torch.int32, device=DEV)
    o, lse = smla.sparse_mla_fwd_paged(torch.empty((0, 32, 512), dtype=torch.bfloat16, device=DEV), cache, table, none,
                                       workspace=ws)
    assert o.shape == (0, 32, 512) and lse.shape == (0, 32)
    smla.cache_alloc(cache, table, none, workspace=ws)
    smla.cache_write(cache, table, none, _i32([0]), torch.empty((0, 512), dtype=torch.bfloat16, device=DEV),
                     workspace=ws)
    assert smla.cache_fork(cache, table, none, none, workspace=ws).shape == (0, 3)
    smla.cache_free(cache, table, workspace=ws)
    smla.cache_free(cache, _i32([[0, -1, -1]]), none, workspace=ws)
    new, count = smla.cache_compact(cache, table, workspace=ws)
    assert new.shape == (0, 3) and (count == 0).all()
    pool.check(cache)


# ------------------------------------------------------------------------------------------------ refusals
def test_tensors_that_a_call_cannot_take():
    smla = _smla()
    from sparse_mla_attention_gb300 import SmlaError, _lib
    pool = Pool(8, 16, 16, seed=19)
    cache = pool.device()
    table, lens = _i32([[0, 1]]), _i32([20])
    q = torch.zeros((1, 16, 512), dtype=torch.bfloat16, device=DEV)
    shifted = torch.zeros(16 * 512 + 1, dtype=torch.bfloat16, device=DEV)[1:].view(1, 16, 512)
    with pytest.raises(SmlaError) as e:
        smla.sparse_mla_fwd_paged(shifted, cache, table, lens)
    assert e.value.code == _lib.SMLA_ERR_ALIGN
    with pytest.raises(SmlaError) as e:
        smla.sparse_mla_fwd_paged(q, cache, table, lens, out=(q, torch.empty((1, 16), device=DEV)))
    assert e.value.code == _lib.SMLA_ERR_OVERLAP
    for bad in (q.cpu(), q.float(), q[0], q.transpose(0, 1)[:, :, ::2]):
        with pytest.raises((ValueError, TypeError)):
            smla.sparse_mla_fwd_paged(bad, cache, table, lens)
    with pytest.raises((ValueError, TypeError)):
        smla.sparse_mla_fwd_paged(q, cache, table.cpu(), lens)
    with pytest.raises((ValueError, TypeError)):
        smla.sparse_mla_fwd_paged(q, cache, table, lens.long())
    with pytest.raises(SmlaError) as e:
        smla.sparse_mla_fwd_paged(torch.zeros((1, 24, 512), dtype=torch.bfloat16, device=DEV), cache, table, lens)
    assert e.value.code == _lib.SMLA_ERR_SHAPE
    with pytest.raises(SmlaError) as e:
        smla.cache_fork(cache, table, lens, _i32([0]), out=table)
    assert e.value.code == _lib.SMLA_ERR_OVERLAP
    with pytest.raises(SmlaError) as e:
        smla.cache_compact(cache, table, out=(torch.empty_like(table), cache.refcount))
    assert e.value.code == _lib.SMLA_ERR_OVERLAP
    with pytest.raises((ValueError, TypeError)):
        smla.cache_write(cache, table, lens, _i32([0, 1]), torch.zeros((1, 512), dtype=torch.float16, device=DEV))
    pool.check(cache)
