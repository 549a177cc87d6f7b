"""GPU tests of accumulated weights, eviction, beam selection and reordering over the paged cache, each against the
64-bit models of decode_reference. Tables, codes, scales, counts, positions and tokens are compared
exactly, sums within the bounds derived there."""

import numpy as np
import pytest
import torch

import cache_reference as R
import decode_reference as M
from test_gpu_cache import DEV, Pool, _i32, _smla, bf16, bf16_dev
from gpu_helpers import to_f64

pytestmark = pytest.mark.gpu


def _f32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(DEV)


def _np(t):
    return t.cpu().numpy()


def _lse(q, pool, table, cu, lens, sink=0.0):
    """fp32 lse [T,H] of the attention, from the model."""
    T, H, _ = q.shape
    out = np.full((T, H), -np.inf, dtype=np.float32)
    for b in range(table.shape[0]):
        for t in range(cu[b], cu[b + 1]):
            if lens[t] == 0:
                continue
            x, _, _ = R.rows_of(pool.codes, pool.scales, table[b], np.arange(lens[t]), pool.page, pool.block)
            s = q[t] @ x.T / np.sqrt(512.0)
            m = s.max(axis=1)
            out[t] = m + np.log(np.exp(s - m[:, None]).sum(axis=1) + np.exp(sink - m))
    return out


def _watch(pool, table, counts, lens, H, decay=1.0, in_place=False, with_cu=True, seed=3, amp=1.0, lse=None):
    smla = _smla()
    rng = np.random.default_rng(seed)
    B, W = table.shape[0], table.shape[1] * pool.page
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    T = int(cu[-1])
    q = bf16(rng.standard_normal((T, H, 512)) * amp)
    if lse is None:
        lse = _lse(q, pool, table, cu, lens)
    earlier = rng.exponential(size=(B, W)).astype(np.float32)
    before = earlier if in_place else np.full((B, W), 7.0, dtype=np.float32)
    cache = pool.device()
    out = _f32(before)
    got = smla.cache_weights(bf16_dev(q), cache, _i32(table), _i32(lens), _f32(lse), out,
                             cu_tokens=_i32(cu) if with_cu else None, earlier=None if in_place else _f32(earlier),
                             decay=decay)
    assert got is out
    ref, bound = M.weights(q, pool.codes, pool.scales, table, cu, lens, lse, earlier, decay, before, pool.page, pool.block)
    got = out.double().cpu().numpy()
    over = np.abs(got - ref) - bound
    assert not np.isnan(over).any()
    assert over.max() <= 0, f"off by {over.max():.3e} over its bound at {np.unravel_index(over.argmax(), over.shape)}"
    pool.check(cache)
    return out


# ------------------------------------------------------------------------------------------------ weights
LENS = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 333]


@pytest.mark.parametrize("H", [16, 32, 48, 64, 80, 96, 112, 128])
@pytest.mark.parametrize("page,block", [(16, 16), (64, 32), (256, 64)])
def test_weights_of_one_token_each(H, page, block):
    pool = Pool(120, page, block, seed=H)
    table = pool.place(LENS)
    pool.fill(table, LENS)
    _watch(pool, table, [1] * len(LENS), LENS, H, with_cu=False)


@pytest.mark.parametrize("decay,in_place", [(0.0, False), (0.0, True), (0.9, False), (0.9, True), (1.0, True),
                                            (-2.0, False)])
def test_weights_with_earlier_ones(decay, in_place):
    pool = Pool(60, 32, 16, seed=1)
    lens = [40, 0, 500, 33]
    table = pool.place(lens)
    pool.fill(table, lens)
    _watch(pool, table, [1] * 4, lens, 48, decay=decay, in_place=in_place)


@pytest.mark.parametrize("H,counts", [(16, [1, 0, 40, 3, 9]), (64, [2, 5, 0, 1, 17]), (128, [3, 1, 1, 4, 7]),
                                      (48, [11, 0, 0, 2, 6])])
@pytest.mark.parametrize("page,block", [(16, 16), (128, 64)])
def test_weights_of_several_tokens(H, counts, page, block):
    pool = Pool(150, page, block, seed=H)
    full = [300, 7, 700, 129, 256]
    table = pool.place(full)
    pool.fill(table, full)
    lens = [max(0, n - c + 1 + i) for n, c in zip(full, counts) for i in range(c)]
    lens[0] = 0                                       # a padded slot
    _watch(pool, table, counts, lens, H)


@pytest.mark.parametrize("H,counts", [(16, [41, 0, 77, 33, 30]), (48, [31, 1, 0, 29, 40]), (64, [0, 60, 0, 0, 0]),
                                      (112, [12, 2, 30, 9, 1]), (128, [9, 1, 40, 0, 5])])
@pytest.mark.parametrize("page,block", [(16, 16), (64, 32), (256, 64)])
def test_weights_of_many_tokens(H, counts, page, block):
    pool = Pool(300, page, block, seed=H)
    full = [300, 67, 1500, 129, 256]
    table = pool.place(full)
    pool.fill(table, full)
    lens = [max(0, n - c + 1 + i) for n, c in zip(full, counts) for i in range(c)]
    lens[3] = 0                                       # a padded slot
    _watch(pool, table, counts, lens, H, decay=0.9)
    _watch(pool, table, counts, lens, H, decay=0.0)


def test_weights_of_many_tokens_with_a_missing_page():
    from sparse_mla_attention_gb300 import SmlaError, _lib
    smla = _smla()
    rng = np.random.default_rng(90)
    pool = Pool(100, 16, 16, seed=91)
    table = pool.place([900, 40])
    pool.fill(table, [900, 40])
    lens, cu = [900 - 39 + i for i in range(40)] + [40], [0, 40, 41]
    q = bf16(rng.standard_normal((41, 64, 512)))
    lse = _lse(q, pool, table, cu, lens)
    bad = table.astype(np.int64).copy()
    bad[0, [0, 30]] = 100, -1
    W = table.shape[1] * 16
    earlier = rng.exponential(size=(2, W)).astype(np.float32)
    out = _f32(np.full((2, W), 7.0))
    with pytest.raises(SmlaError) as e:
        smla.cache_weights(bf16_dev(q), pool.device(), _i32(bad), _i32(lens), _f32(lse), out, cu_tokens=_i32(cu),
                           earlier=_f32(earlier), decay=0.5)
    assert e.value.code == _lib.SMLA_ERR_INDEX
    ref, bound = M.weights(q, pool.codes, pool.scales, table, cu, lens, lse, earlier, 0.5,
                           np.full((2, W), 7.0, dtype=np.float32), 16, 16)
    for p in (0, 480):                                # (halving is exact)
        ref[0, p:p + 16], bound[0, p:p + 16] = 0.5 * earlier[0, p:p + 16], 0.0
    assert (np.abs(out.double().cpu().numpy() - ref) <= bound).all()


def test_weights_of_a_long_sequence_and_many_short_ones():
    lens = [20000] + list(range(1, 120))
    pool = Pool(1200, 64, 64, seed=4)
    table = pool.place(lens, extra=3)
    pool.fill(table, lens)
    _watch(pool, table, [1] * len(lens), lens, 64)


def test_weights_of_many_tokens_over_many_tiles():
    pool = Pool(200, 64, 32, seed=5)
    full = [3000, 5000]
    table = pool.place(full)
    pool.fill(table, full)
    counts = [33, 20]
    lens = [n - c + 1 + i for n, c in zip(full, counts) for i in range(c)]
    _watch(pool, table, counts, lens, 96, decay=0.0)


def test_weights_for_scales_of_every_size_and_scores_far_apart():
    rng = np.random.default_rng(6)
    pool = Pool(60, 64, 16, seed=7, junk=False)
    lens = [700, 64, 1, 900]
    table = pool.place(lens)
    pool.codes[:] = R.encode(rng.standard_normal(pool.codes.shape) * 30)
    pool.scales[:] = np.exp2(rng.integers(-30, -4, size=pool.scales.shape))
    _watch(pool, table, [1] * 4, lens, 64, amp=6.0)


def test_weights_of_heads_that_saw_nothing_and_of_odd_values():
    smla = _smla()
    rng = np.random.default_rng(8)
    pool = Pool(20, 16, 16, seed=9)
    lens = [50, 20, 33]
    table = pool.place(lens)
    pool.fill(table, lens)
    q = bf16(rng.standard_normal((3, 32, 512)))
    lse = _lse(q, pool, table, [0, 1, 2, 3], lens)
    lse[0, 5] = -np.inf
    q[1, 3, 100] = np.nan
    q[2, 4, 7] = np.inf
    W = table.shape[1] * 16
    out = torch.zeros((3, W), device=DEV)
    smla.cache_weights(bf16_dev(q), pool.device(), _i32(table), _i32(lens), _f32(lse), out)
    got = out.double().cpu().numpy()
    ref, bound = M.weights(q[:1], pool.codes, pool.scales, table[:1], [0, 1], lens[:1], lse[:1], np.zeros((1, W)), 0.0,
                           np.zeros((1, W), dtype=np.float32), 16, 16)
    assert (np.abs(got[0] - ref[0]) <= bound[0]).all()
    for b in (1, 2):                                   # NaN where the head looks, nowhere else
        assert np.isnan(got[b, : lens[b]]).all() and (got[b, lens[b]:] == 0).all()


def test_weights_with_bad_indices_are_reported():
    from sparse_mla_attention_gb300 import SmlaError, _lib
    smla = _smla()
    rng = np.random.default_rng(10)
    pool = Pool(30, 16, 16, seed=11)
    lens = [60, 45, 30]
    table = pool.place(lens)
    pool.fill(table, lens)
    q = bf16(rng.standard_normal((3, 16, 512)))
    W = table.shape[1] * 16
    lse = _lse(q, pool, table, [0, 1, 2, 3], lens)
    ws = smla.Workspace(DEV)

    def call(table, lens, cu):
        out = torch.zeros((3, W), device=DEV)
        with pytest.raises(SmlaError) as e:
            smla.cache_weights(bf16_dev(q), pool.device(), _i32(table), _i32(lens), _f32(lse), out, cu_tokens=_i32(cu),
                               workspace=ws)
        assert e.value.code == _lib.SMLA_ERR_INDEX
        return out.double().cpu().numpy()

    ref, bound = M.weights(q, pool.codes, pool.scales, table, [0, 1, 2, 3], lens, lse, np.zeros((3, W)), 0.0,
                           np.zeros((3, W), dtype=np.float32), 16, 16)
    for page in (-1, 30, 1 << 30, -(1 << 31)):
        bad = table.astype(np.int64).copy()
        bad[1, 1] = page
        got = call(bad, lens, [0, 1, 2, 3])
        live = np.ones((3, W), dtype=bool)
        live[1, 16:32] = False
        assert (np.abs(got - ref)[live] <= bound[live]).all() and (got[~live] == 0).all()
    for cu, dead in (([0, 1, 4, 3], [1, 2]), ([0, 2, 1, 3], [1]), ([-1, 1, 2, 3], [0])):
        got = call(table, lens, cu)
        for b in dead:
            assert (got[b] == 0).all()
    got = call(table, [60, 45, -5], [0, 1, 2, 3])
    assert (got[2] == 0).all() and (np.abs(got - ref)[:2] <= bound[:2]).all()


def test_weights_do_not_depend_on_the_run():
    smla = _smla()
    pool = Pool(400, 64, 32, seed=12)
    lens = [9001, 4000, 77]
    table = pool.place(lens)
    pool.fill(table, lens)
    cache = pool.device()
    rng = np.random.default_rng(13)
    q, lse = bf16_dev(rng.standard_normal((3, 128, 512))), _f32(rng.standard_normal((3, 128)) + 9)
    runs = []
    for _ in range(3):
        out = torch.zeros((3, table.shape[1] * 64), device=DEV)
        runs.append(smla.cache_weights(q, cache, _i32(table), _i32(lens), lse, out))
    assert torch.equal(runs[0], runs[1]) and torch.equal(runs[0], runs[2])


# ------------------------------------------------------------------------------------------------ eviction
def _evict_and_check(pool, table, lens, w, keep, first=0, recent=0):
    smla = _smla()
    cache = pool.device()
    tt, lt, wt = _i32(table), _i32(lens), _f32(w)
    got = smla.cache_evict(cache, tt, lt, wt, keep, first=first, recent=recent)
    ref = M.evict(pool.codes, pool.scales, pool.refcount, table, lens, w, keep, first, recent, pool.page, pool.block)
    for name, g, r in zip(("table", "lens", "weights", "kept"), got, ref):
        np.testing.assert_array_equal(_np(g), r, err_msg=name)
    pool.check(cache)
    np.testing.assert_array_equal(_np(tt), table)
    np.testing.assert_array_equal(_np(lt), lens)
    np.testing.assert_array_equal(_np(wt), w)
    return cache, got


def _heavy(rng, B, W, ties=0.3):
    w = np.exp(2 * rng.standard_normal((B, W))).astype(np.float32)
    w[rng.random((B, W)) < ties] = 0.0
    w[rng.random((B, W)) < ties] = 1.5
    return w


@pytest.mark.parametrize("page,block", [(16, 16), (64, 16), (64, 64), (128, 32), (256, 64)])
@pytest.mark.parametrize("keep,first,recent", [(1, 0, 0), (1, 1, 0), (64, 3, 10), (100, 0, 100), (100, 40, 60),
                                               (333, 4, 32)])
def test_evict_matches_the_model(page, block, keep, first, recent):
    rng = np.random.default_rng(page + keep)
    lens = [0, 1, 2, 63, 64, 65, 100, 101, 333, 700]
    pool = Pool(300, page, block, seed=14)
    table = pool.place(lens, extra=2)
    pool.fill(table, lens)
    _evict_and_check(pool, table, lens, _heavy(rng, len(lens), table.shape[1] * page), keep, first, recent)


@pytest.mark.parametrize("lens,keep", [([40000, 20001, 300], 12345), ([90001], 1000), ([17000, 16384, 16385], 16383)])
def test_evict_long_sequences(lens, keep):
    rng = np.random.default_rng(keep)
    pool = Pool(2400, 64, 32, seed=15, junk=False)
    table = pool.place(lens)
    _evict_and_check(pool, table, lens, _heavy(rng, len(lens), table.shape[1] * 64), keep, 4, 64)


def test_evict_by_odd_weights():
    rng = np.random.default_rng(16)
    lens = [400, 400, 400, 400, 400]
    pool = Pool(100, 32, 32, seed=17, junk=False)
    table = pool.place(lens)
    w = rng.standard_normal((5, table.shape[1] * 32)).astype(np.float32)
    w[0] = 1.0                                         # ties alone
    w[1, ::2], w[1, 1::2] = 0.0, -0.0
    w[2, rng.random(w.shape[1]) < 0.5] = np.nan
    w[3, rng.random(w.shape[1]) < 0.2] = np.inf
    w[3, rng.random(w.shape[1]) < 0.4] = -np.inf
    w[4] = np.nan
    smla = _smla()
    cache = pool.device()
    got = smla.cache_evict(cache, _i32(table), _i32(lens), _f32(w), 150, first=2, recent=7)
    ref = M.evict(pool.codes, pool.scales, pool.refcount, table, lens, w, 150, 2, 7, 32, 32)
    np.testing.assert_array_equal(_np(got[3]), ref[3])
    np.testing.assert_array_equal(_np(got[2]), ref[2])
    np.testing.assert_array_equal(_np(got[0]), ref[0])
    pool.check(cache)


def _crowded(rng, shape, kind):
    """Weights that differ in their last bits only: all in one of the 2048 widest bins (kind 21), all alike but for 10
    bits (kind 10), or half and half, so that the last one to stay can be in either."""
    bits = np.float32(1.0).view(np.int32) + rng.integers(0, 1 << min(kind, 21), size=shape)
    if kind == 22:
        low = rng.random(shape) < 0.5
        bits[low] = np.float32(0.75).view(np.int32) + rng.integers(0, 1 << 10, size=int(low.sum()))
    return bits.astype(np.int32).view(np.float32)


@pytest.mark.parametrize("kind", [10, 21, 22])
@pytest.mark.parametrize("lens,keep", [([16384, 9000, 5000, 4097], 1), ([16000, 8300, 5000, 4100], 2500),
                                       ([16384, 16383, 12001], 8191), ([60000, 30001], 11111), ([140003, 131072], 70001),
                                       ([140003], 9)])
def test_evict_by_crowded_weights(lens, keep, kind):
    rng = np.random.default_rng(keep + kind)
    pool = Pool(7000, 64, 64, seed=38, junk=False)
    table = pool.place(lens)
    _evict_and_check(pool, table, lens, _crowded(rng, (len(lens), table.shape[1] * 64), kind), keep, 0, 0)
    w = -_crowded(rng, (len(lens), table.shape[1] * 64), kind)
    w[:, 5::7] = np.nan
    pool = Pool(7000, 64, 64, seed=39, junk=False)
    table = pool.place(lens)
    _evict_and_check(pool, table, lens, w, keep, min(keep, 3), 0)


def test_evict_many_sequences():
    rng = np.random.default_rng(18)
    lens = rng.integers(0, 200, size=700)
    pool = Pool(10000, 16, 16, seed=19, junk=False)
    table = pool.place(lens)
    _evict_and_check(pool, table, lens, _heavy(rng, 700, table.shape[1] * 16), 70, 1, 20)


def test_evict_with_too_few_pages_changes_nothing():
    from sparse_mla_attention_gb300 import SmlaError, _lib
    smla = _smla()
    rng = np.random.default_rng(20)
    lens = [100, 80, 60]
    for spare, enough in ((9, True), (8, False)):
        pool = Pool(7 + 5 + 4 + spare, 16, 16, seed=21)
        table = pool.place(lens)
        pool.fill(table, lens)
        w = _heavy(rng, 3, table.shape[1] * 16)
        if enough:                                     # 4 + 4 + 4 of 64 positions need 12, of 48 positions 9
            _evict_and_check(pool, table, lens, w, 48)
            continue
        cache = pool.device()
        out = (_i32(table), _i32(lens), _f32(w), _i32(np.zeros((3, 48))))
        with pytest.raises(SmlaError) as e:
            smla.cache_evict(cache, _i32(table), _i32(lens), _f32(w), 48, out=out)
        assert e.value.code == _lib.SMLA_ERR_PAGES
        assert (out[0] == -1).all() and (out[1] == 0).all()
        pool.check(cache)


def test_evict_with_bad_pages_and_lengths_is_reported():
    from sparse_mla_attention_gb300 import SmlaError, _lib
    smla = _smla()
    rng = np.random.default_rng(22)
    lens = [100, 80]
    pool = Pool(40, 16, 16, seed=23)
    table = pool.place(lens)
    pool.fill(table, lens)
    w = _heavy(rng, 2, table.shape[1] * 16)
    bad = table.astype(np.int64).copy()
    bad[0, 2], bad[1, 0] = 40, -(1 << 31)
    cache = pool.device()
    ws = smla.Workspace(DEV)
    out = (_i32(table), _i32(lens), _f32(w), _i32(np.zeros((2, 64))))
    with pytest.raises(SmlaError) as e:
        smla.cache_evict(cache, _i32(bad), _i32(lens), _f32(w), 64, first=40, workspace=ws, out=out)
    assert e.value.code == _lib.SMLA_ERR_INDEX
    ref = M.evict(pool.codes, pool.scales, pool.refcount, bad, lens, w, 64, 40, 0, 16, 16)
    np.testing.assert_array_equal(_np(out[0]), ref[0])
    pool.check(cache)
    # lengths beyond the table or below zero are clamped
    pool = Pool(40, 16, 16, seed=24, junk=False)
    table = pool.place([128, 128], extra=0)
    cache = pool.device()
    w = _heavy(rng, 2, 128)
    out = (_i32(table), _i32([0, 0]), _f32(w), _i32(np.zeros((2, 30))))
    with pytest.raises(SmlaError) as e:
        smla.cache_evict(cache, _i32(table), _i32([1 << 30, -3]), _f32(w), 30, workspace=ws, out=out)
    assert e.value.code == _lib.SMLA_ERR_INDEX
    ref = M.evict(pool.codes, pool.scales, pool.refcount, table, [128, 0], w, 30, 0, 0, 16, 16)
    for g, r in zip(out, ref):
        np.testing.assert_array_equal(_np(g), r)
    pool.check(cache)


# ------------------------------------------------------------------------------------------------ beams
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def _select_and_check(x, scores, n, done=None, eos=-1):
    """x: logits tensor on the GPU, of any stride."""
    smla = _smla()
    got = smla.beam_select(x, _f32(scores), n=n, done=None if done is None else torch.from_numpy(done).to(DEV), eos=eos)
    s32 = scores.astype(np.float32).astype(np.float64)
    ref = M.select(x.double().cpu().numpy(), s32, n, done, eos)
    np.testing.assert_array_equal(_np(got[0]), ref[0])
    np.testing.assert_array_equal(_np(got[1]), ref[1])
    fine = np.isfinite(ref[2])
    s = got[2].double().cpu().numpy()
    assert (s[~fine] == -np.inf).all()
    # one rounding to fp32, and the sum of exponentials: 33 terms and their exponentials in fp32, arguments of up to 100
    # with a rounding before and behind the factor log2(e)
    bound = 2.0 ** -24 * np.abs(ref[2][fine]) + 300 * 2.0 ** -24
    assert (np.abs(s[fine] - ref[2][fine]) <= bound).all()
    return got


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,K,V,n", [(1, 1, 1, 1), (1, 1, 5, 8), (3, 2, 100, 2), (2, 4, 8191, 4), (2, 3, 8192, 7),
                                     (1, 8, 8200, 16), (2, 5, 50001, 10), (1, 64, 3000, 64), (5, 1, 16400, 33),
                                     (1, 2, 131072, 8), (40, 3, 777, 3)])
def test_select_matches_the_model(dtype, B, K, V, n):
    g = torch.Generator(device=DEV).manual_seed(B * K + V)
    x = (torch.randn(B * K, V, generator=g, device=DEV) * 3).to(dtype)
    rng = np.random.default_rng(V)
    _select_and_check(x, -np.abs(rng.standard_normal((B, K))) * 3, n)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,lead", [(0, 0), (1, 0), (3, 1), (8, 5), (64, 3), (5, 7)])
def test_select_of_rows_that_start_anywhere(dtype, pad, lead):
    g = torch.Generator(device=DEV).manual_seed(pad * 8 + lead)
    wide = (torch.randn(6, 9000 + lead + pad, generator=g, device=DEV) * 3)
    wide[:, :lead], wide[:, lead + 9000:] = 100.0, 100.0                 # (not to be seen)
    x = wide.to(dtype)[:, lead:lead + 9000]
    _select_and_check(x, np.zeros((2, 3)), 9)
    _select_and_check(x[:, :3], np.zeros((2, 3)), 9)


def test_select_of_ended_dead_and_banned_beams():
    g = torch.Generator(device=DEV).manual_seed(1)
    V = 20000
    x = torch.randn(24, V, generator=g, device=DEV) * 3
    x[torch.rand(24, V, generator=g, device=DEV) < 0.4] = -float("inf")
    x[2] = -float("inf")                              # nothing allowed
    x[3, 77] = float("nan")
    x[5, 19999] = float("inf")
    x[6, 1:] = -float("inf")                          # one token allowed
    x[20:24] = -float("inf")                          # a group without a candidate
    scores = -np.abs(np.random.default_rng(2).standard_normal((6, 4)))
    scores[1] = [-np.inf, np.nan, np.inf, -1.0]
    done = np.zeros((6, 4), dtype=bool)
    done[0, 0] = done[2] = done[3, 1] = True
    scores[3, 1] = -np.inf                            # ended, and dead
    for n in (1, 4, 12):
        _select_and_check(x, scores, n, done, eos=5)
        _select_and_check(x.to(torch.bfloat16), scores, n)


@pytest.mark.parametrize("dtype", TYPES)
def test_select_with_ties(dtype):
    V = 40000
    x = torch.zeros(8, V, device=DEV)
    x[1, V // 2:] = 1.0
    x[2, ::3] = 2.0
    x[3] = torch.arange(V, device=DEV) / V            # ascending (in 16 bits with many ties)
    x[4] = -torch.arange(V, device=DEV) / V
    x[5, 100:] = -float("inf")
    x[6, ::2] = -0.0
    x[7] = x[3]
    x = x.to(dtype)
    for n in (1, 5, 64):
        _select_and_check(x, np.zeros((4, 2)), n)
        _select_and_check(x[3:8].repeat_interleave(2, 0)[1:9], np.zeros((1, 8)), n)


def test_select_of_peaked_rows():
    # nearly all weight on one token, and logits far below it
    x = torch.full((4, 30000), -60000.0, device=DEV)
    x[0, 29999] = 60000.0
    x[1, 0] = -59990.0
    x[2] = torch.linspace(-80, 20, 30000, device=DEV)
    x[3, 12345] = 3e38
    _select_and_check(x[:3], np.array([[-1.0, -2.0, -0.5]]), 6)
    _select_and_check(x[2:], np.array([[-1.0, -2.0]]), 3)


# ------------------------------------------------------------------------------------------------ reordering
def _reorder_and_check(pool, table, lens, parents, w=None):
    smla = _smla()
    cache = pool.device()
    got = smla.cache_reorder(cache, _i32(table), _i32(lens), _i32(parents), weights=None if w is None else _f32(w))
    ref = M.reorder(pool.codes, pool.scales, pool.refcount, table, lens, parents, pool.page, w)
    np.testing.assert_array_equal(_np(got[0]), ref[0])
    np.testing.assert_array_equal(_np(got[1]), ref[1])
    if w is not None:
        np.testing.assert_array_equal(_np(got[2]), ref[2])
    pool.check(cache)
    return cache, got, ref


@pytest.mark.parametrize("page,block", [(16, 16), (64, 32), (256, 64)])
@pytest.mark.parametrize("weights", [False, True])
def test_reorder_matches_the_model(page, block, weights):
    rng = np.random.default_rng(page)
    lens = [0, 1, 15, 16, 17, 64, 100, 256, 300, 513]
    pool = Pool(120, page, block, seed=30)
    table = pool.place(lens, extra=2)
    pool.fill(table, lens)
    w = rng.exponential(size=(len(lens), table.shape[1] * page)).astype(np.float32) if weights else None
    for step in range(6):
        parents = rng.choice([-1] + list(range(len(lens))), size=rng.integers(1, 14))
        _, got, ref = _reorder_and_check(pool, table, lens, parents, w)
        table, lens, w = ref
        held = np.bincount(table[table >= 0], minlength=pool.num_pages)
        np.testing.assert_array_equal(held, pool.refcount)


def test_reorder_of_many_beams_and_shared_prompts():
    rng = np.random.default_rng(31)
    groups, K, page = 60, 8, 16
    lens = np.repeat(rng.integers(20, 400, size=groups), K)
    pool = Pool(9000, page, 16, seed=32, junk=False)
    table = pool.place(lens)
    for b in range(groups * K):                       # the first page of a group is shared
        lead = b // K * K
        if b != lead:
            pool.refcount[table[b, 0]] = 0
            table[b, 0] = table[lead, 0]
            pool.refcount[table[lead, 0]] += 1
    w = rng.exponential(size=(groups * K, table.shape[1] * page)).astype(np.float32)
    parents = np.concatenate([g * K + rng.integers(0, K, size=K) for g in range(groups)])
    _reorder_and_check(pool, table, lens, parents, w)


def test_reorder_in_a_full_pool_takes_the_last_pages_of_ended_rows():
    from sparse_mla_attention_gb300 import SmlaError, _lib
    smla = _smla()
    lens = [20, 25, 17, 31]
    pool = Pool(8, 16, 16, seed=33)
    table = pool.place(lens, extra=0)
    pool.fill(table, lens)
    _, _, ref = _reorder_and_check(pool, table, lens, [2, 2, 0, 2])
    assert (pool.refcount > 0).sum() == 6             # two first pages came free
    table, lens, _ = ref
    # short of a page: nothing changes (a child of each and three copies; two pages are free, no row ends)
    cache = pool.device()
    out = (_i32(np.zeros((7, 2))), _i32(np.zeros(7)), None)
    with pytest.raises(SmlaError) as e:
        smla.cache_reorder(cache, _i32(table), _i32(lens), _i32([0, 1, 2, 3, 3, 3, 3]), out=out)
    assert e.value.code == _lib.SMLA_ERR_PAGES
    assert (out[0] == -1).all() and (out[1] == 0).all()
    pool.check(cache)


def test_reorder_with_bad_rows_is_reported():
    from sparse_mla_attention_gb300 import SmlaError, _lib
    smla = _smla()
    lens = [40, 20, 33]
    ws = smla.Workspace(DEV)

    def call(pool, table, lens, parents, code):
        cache = pool.device()
        out = (_i32(np.zeros((len(parents), table.shape[1]))), _i32(np.zeros(len(parents))), None)
        with pytest.raises(SmlaError) as e:
            smla.cache_reorder(cache, _i32(table), _i32(lens), _i32(parents), out=out, workspace=ws)
        assert e.value.code == code
        return cache, out

    pool = Pool(30, 16, 16, seed=34)
    table = pool.place(lens)
    cache, out = call(pool, table, lens, [0, 3, -2, 1, 2], _lib.SMLA_ERR_INDEX)
    ref = M.reorder(pool.codes, pool.scales, pool.refcount, table, lens, [0, -1, -1, 1, 2], 16)
    np.testing.assert_array_equal(_np(out[0]), ref[0])
    np.testing.assert_array_equal(_np(out[1]), ref[1])
    pool.check(cache)
    # a page out of range: left out for the child that would share it, and not given back
    pool = Pool(30, 16, 16, seed=35)
    table = pool.place(lens)
    bad = table.astype(np.int64).copy()
    bad[0, 1], bad[1, 0] = 30, -(1 << 31)
    pool.refcount[[table[0, 1], table[1, 0]]] = 0
    cache, out = call(pool, bad, lens, [0, 0, 2], _lib.SMLA_ERR_INDEX)
    got = _np(out[0])
    assert got[0, 1] == 30 and got[1, 1] == -1 and got[1, 0] == table[0, 0]
    assert _np(cache.refcount)[table[0, 0]] == 2
    # a count that is zero already
    pool = Pool(30, 16, 16, seed=36)
    table = pool.place(lens)
    pool.refcount[[table[0, 0], table[1, 0]]] = 0
    cache, out = call(pool, table, lens, [0, 0, 2], _lib.SMLA_ERR_REFCOUNT)
    assert _np(out[0])[1, 0] == -1 and (_np(cache.refcount) >= 0).all()


# ------------------------------------------------------------------------------------------------ together
def test_a_sequence_is_evicted_as_it_decodes():
    """alloc, write, attend, accumulate, evict: captured step by step with a budget, against the models."""
    smla = _smla()
    page, block, H, B, keep = 16, 16, 32, 3, 40
    rng = np.random.default_rng(40)
    pool = Pool(80, page, block, seed=41)
    lens = np.array([47, 30, 3], dtype=np.int32)
    width = 6
    table = np.full((B, width), -1, dtype=np.int32)
    cache = pool.device()
    tt, start, end = _i32(table), _i32(np.zeros(B)), _i32(lens)
    ws = smla.Workspace(DEV)
    ws.get(64 << 20)
    kw = dict(workspace=ws, check_status=False)
    smla.cache_alloc(cache, tt, end, workspace=ws)
    R.alloc(pool.refcount, table, lens, page)
    cu = np.concatenate([[0], np.cumsum(lens)])
    rows = bf16(rng.standard_normal((cu[-1], 512)))
    smla.cache_write(cache, tt, start, _i32(cu), bf16_dev(rows), workspace=ws)
    R.write(pool.codes, pool.scales, table, np.zeros(B, dtype=int), cu, rows, page, block)

    one, row_t, q_t = _i32(np.arange(B + 1)), bf16_dev(np.zeros((B, 512))), bf16_dev(np.zeros((B, H, 512)))
    o, lse = torch.empty((B, H, 512), dtype=torch.bfloat16, device=DEV), torch.empty((B, H), device=DEV)
    acc = torch.zeros((B, width * page), device=DEV)
    new = (_i32(np.full((B, width), -1)), _i32(np.zeros(B)), torch.zeros_like(acc), _i32(np.zeros((B, keep))))

    def step():
        smla.cache_alloc(cache, tt, end, **kw)
        smla.cache_write(cache, tt, start, one, row_t, **kw)
        smla.sparse_mla_fwd_paged(q_t, cache, tt, end, out=(o, lse), **kw)
        smla.cache_weights(q_t, cache, tt, end, lse, acc, decay=0.9, **kw)

    def evict():
        smla.cache_evict(cache, tt, end, acc, keep, first=2, recent=5, out=new, **kw)
        smla.cache_free(cache, tt, **kw)
        tt.copy_(new[0]); end.copy_(new[1]); acc.copy_(new[2])
    graphs = []
    for f in (step, evict):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f()
        graphs.append(g)
    for i in range(12):
        row, q = bf16(rng.standard_normal((B, 512)) * (1 + i % 3)), bf16(rng.standard_normal((B, H, 512)))
        start.copy_(_i32(lens)); lens = lens + 1; end.copy_(_i32(lens))
        row_t.copy_(bf16_dev(row)); q_t.copy_(bf16_dev(q))
        was = acc.cpu().numpy()
        graphs[0].replay()
        assert R.alloc(pool.refcount, table, lens, page)
        R.write(pool.codes, pool.scales, table, lens - 1, np.arange(B + 1), row, page, block)
        ref, _, ob, _ = R.attend(q, pool.codes, pool.scales, table, lens, page, block)
        assert (np.abs(to_f64(o) - ref) <= ob).all()
        w, bound = M.weights(q, pool.codes, pool.scales, table, np.arange(B + 1), lens, lse.cpu().numpy(), was, 0.9, was,
                             page, block)
        assert (np.abs(acc.double().cpu().numpy() - w) <= bound).all()
        if i % 4 == 3:
            w = acc.cpu().numpy()
            graphs[1].replay()
            n_table, lens, n_w, kept = M.evict(pool.codes, pool.scales, pool.refcount, table, lens, w, keep, 2, 5, page,
                                               block)
            R.free_rows(pool.refcount, table, range(B))
            table = n_table
            np.testing.assert_array_equal(new[3].cpu().numpy(), kept)
            np.testing.assert_array_equal(acc.cpu().numpy(), n_w)
        np.testing.assert_array_equal(tt.cpu().numpy(), table)
        np.testing.assert_array_equal(end.cpu().numpy(), lens)
        pool.check(cache)


def test_beams_go_on_with_their_sequences():
    """select, reorder, alloc, write, attend, step after step, in a captured graph with two tables in turn."""
    smla = _smla()
    page, block, H, groups, K, V = 16, 16, 16, 2, 3, 500
    B, width = groups * K, 5
    rng = np.random.default_rng(50)
    pool = Pool(40, page, block, seed=51)
    lens = np.array([13] * K + [29] * K, dtype=np.int32)
    table = np.full((B, width), -1, dtype=np.int32)
    cache = pool.device()
    ws = smla.Workspace(DEV)
    ws.get(64 << 20)
    kw = dict(workspace=ws, check_status=False)
    tables, ends = [_i32(table), _i32(table)], [_i32(lens), _i32(lens)]
    smla.cache_alloc(cache, tables[0], ends[0], workspace=ws)
    R.alloc(pool.refcount, table, lens, page)
    cu = np.concatenate([[0], np.cumsum(lens)])
    rows = bf16(rng.standard_normal((cu[-1], 512)))
    smla.cache_write(cache, tables[0], _i32(np.zeros(B)), _i32(cu), bf16_dev(rows), workspace=ws)
    R.write(pool.codes, pool.scales, table, np.zeros(B, dtype=int), cu, rows, page, block)
    one, row_t, q_t = _i32(np.arange(B + 1)), bf16_dev(np.zeros((B, 512))), bf16_dev(np.zeros((B, H, 512)))
    o, lse = torch.empty((B, H, 512), dtype=torch.bfloat16, device=DEV), torch.empty((B, H), device=DEV)
    logits = torch.zeros((B, V), dtype=torch.bfloat16, device=DEV)
    scores = torch.zeros((groups, K), device=DEV)
    picked = tuple(torch.zeros((groups, K), dtype=d, device=DEV) for d in (torch.int32, torch.int32, torch.float32))
    after = _i32(lens)

    def step(k):
        def f():
            smla.beam_select(logits, scores, workspace=ws, out=picked)
            scores.copy_(picked[2])
            smla.cache_reorder(cache, tables[k], ends[k], picked[0].view(-1), out=(tables[1 - k], ends[1 - k], None),
                               **kw)
            after.copy_(ends[1 - k] + 1)
            smla.cache_alloc(cache, tables[1 - k], after, **kw)
            smla.cache_write(cache, tables[1 - k], ends[1 - k], one, row_t, **kw)
            ends[1 - k].copy_(after)
            smla.sparse_mla_fwd_paged(q_t, cache, tables[1 - k], ends[1 - k], out=(o, lse), **kw)
        return f
    graphs = []
    for k in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(k)()
        graphs.append(g)
    s = np.zeros((groups, K))
    for i in range(8):
        x = bf16(rng.standard_normal((B, V)) * 2)
        row, q = bf16(rng.standard_normal((B, 512))), bf16(rng.standard_normal((B, H, 512)))
        logits.copy_(bf16_dev(x)); row_t.copy_(bf16_dev(row)); q_t.copy_(bf16_dev(q))
        graphs[i & 1].replay()
        parents, tokens, _ = M.select(x, s, K)
        np.testing.assert_array_equal(_np(picked[0]), parents)
        np.testing.assert_array_equal(_np(picked[1]), tokens)
        s = picked[2].double().cpu().numpy()
        table, lens, _ = M.reorder(pool.codes, pool.scales, pool.refcount, table, lens, parents.reshape(-1), page)
        assert R.alloc(pool.refcount, table, lens + 1, page)
        R.write(pool.codes, pool.scales, table, lens, np.arange(B + 1), row, page, block)
        lens = lens + 1
        np.testing.assert_array_equal(_np(tables[1 - (i & 1)]), table)
        ref, _, ob, _ = R.attend(q, pool.codes, pool.scales, table, lens, page, block)
        assert (np.abs(to_f64(o) - ref) <= ob).all()
        pool.check(cache)


@pytest.mark.parametrize("fill", [False, True])      # random codes (nearly every row has a NaN among them), or rows
def test_decode_calls_at_once_on_two_streams(fill):
    smla = _smla()
    rng = np.random.default_rng(60)
    page, block, H = 64, 32, 64
    lens = [3000, 100, 1, 0, 777]
    pools, work = [], []
    for k in range(2):
        pool = Pool(300, page, block, seed=61 + k, junk=False)
        table = pool.place(lens)
        pools.append((pool, table))
        if fill:
            pool.fill(table, lens)
        cache = pool.device()
        q = bf16_dev(rng.standard_normal((5, H, 512)))
        x = torch.randn(8, 30000, device=DEV)
        work.append((cache, _i32(table), _i32(lens), q, x, _f32(rng.exponential(size=(5, table.shape[1] * page))),
                     smla.Workspace(DEV)))
    scores = torch.zeros((2, 4), device=DEV)

    def once(cache, table, lens, q, x, w, ws):
        lse = torch.full((5, H), 9.0, device=DEV)
        out = smla.cache_weights(q, cache, table, lens, lse, torch.zeros_like(w), earlier=w, workspace=ws,
                                 check_status=False)
        new = smla.cache_evict(cache, table, lens, out, 128, first=4, recent=32, workspace=ws, check_status=False)
        smla.cache_free(cache, new[0].clone(), workspace=ws, check_status=False)
        return (out, *new, *smla.beam_select(x, scores, workspace=ws))
    alone = [once(*w) for w in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for i in range(8):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k].append(once(*work[k]))
    torch.cuda.synchronize()
    for k in range(2):
        for run in got[k]:
            assert all(torch.equal(a.view(torch.int32), b.view(torch.int32)) for a, b in zip(run, alone[k]))


def test_empty_decode_batches():
    smla = _smla()
    pool = Pool(8, 16, 16, seed=70)
    cache = pool.device()
    ws = smla.Workspace(DEV)
    none, table = _i32([]), torch.empty((0, 3), dtype=torch.int32, device=DEV)
    w = torch.empty((0, 48), device=DEV)
    q, lse = torch.empty((0, 32, 512), dtype=torch.bfloat16, device=DEV), torch.empty((0, 32), device=DEV)
    smla.cache_weights(q, cache, table, none, lse, w, workspace=ws)
    out = torch.full((2, 48), 3.0, device=DEV)
    smla.cache_weights(q, cache, _i32(np.full((2, 3), -1)), none, lse, out, cu_tokens=_i32([0, 0, 0]), workspace=ws)
    assert (out == 3.0).all()
    new = smla.cache_evict(cache, table, none, w, 5, workspace=ws)
    assert new[0].shape == (0, 3) and new[3].shape == (0, 5)
    new = smla.cache_reorder(cache, table, none, none, weights=w, workspace=ws)
    assert new[0].shape == (0, 3) and new[2].shape == (0, 48)
    new = smla.cache_reorder(cache, table, none, _i32([-1, -1]), weights=w, workspace=ws)
    assert (new[0] == -1).all() and (new[1] == 0).all() and (new[2] == 0).all()
    smla.cache_reorder(cache, _i32(np.full((2, 3), -1)), _i32([0, 0]), none, workspace=ws)
    p, t, s = smla.beam_select(torch.empty((0, 9), device=DEV), torch.empty((0, 4), device=DEV), workspace=ws)
    assert p.shape == t.shape == s.shape == (0, 4)
    pool.check(cache)


def test_memory_behind_the_decode_outputs_stays():
    smla = _smla()
    rng = np.random.default_rng(71)
    lens = [300, 20]
    pool = Pool(60, 16, 16, seed=72)
    table = pool.place(lens)
    pool.fill(table, lens)
    cache = pool.device()
    W = table.shape[1] * 16
    big = [torch.full((3 * k,), 7, dtype=d, device=DEV) for k, d in
           ((2 * table.shape[1], torch.int32), (2, torch.int32), (2 * W, torch.float32), (2 * 50, torch.int32))]
    out = (big[0][:2 * table.shape[1]].view(2, -1), big[1][:2], big[2][:2 * W].view(2, -1), big[3][:100].view(2, 50))
    w = _f32(_heavy(rng, 2, W))
    smla.cache_evict(cache, _i32(table), _i32(lens), w, 50, out=out)
    smla.cache_free(cache, out[0].clone())
    x = torch.randn(6, 9001, device=DEV)
    picks = [torch.full((20,), 7, dtype=d, device=DEV) for d in (torch.int32, torch.int32, torch.float32)]
    smla.beam_select(x, torch.zeros((2, 3), device=DEV), n=5, out=tuple(p[:10].view(2, 5) for p in picks))
    for t, k in zip(big + picks, (2 * table.shape[1], 2, 2 * W, 100, 10, 10, 10)):
        assert (t[k:] == 7).all()


def test_reorder_of_more_rows_than_one_block_plans():
    rng = np.random.default_rng(80)
    for B, n in ((5000, 5000), (3, 20000)):
        lens = rng.integers(0, 40, size=B)
        pool = Pool(int((-(-lens // 16)).sum()) + n + 10, 16, 16, seed=81, junk=False)
        table = pool.place(lens)
        _reorder_and_check(pool, table, lens, rng.integers(-1, B, size=n))


def test_select_of_more_candidates_than_one_batch():
    rng = np.random.default_rng(82)
    x = torch.randn(64, 60000, device=DEV)
    _select_and_check(x, rng.standard_normal((1, 64)), 64)
    x = torch.sort(torch.randn(6, 200000, device=DEV), dim=1)[0]
    _select_and_check(x, rng.standard_normal((2, 3)), 64)
    _select_and_check(x.flip(1).half(), rng.standard_normal((2, 3)), 17)


@pytest.mark.parametrize("H,tokens,n", [(128, 300, 300), (16, 700, 130), (48, 211, 5), (64, 150, 2000)])
def test_weights_of_whole_prompts(H, tokens, n):
    # few tiles and many tokens: every processor has a part of a tile
    pool = Pool(100, 32, 32, seed=H)
    table = pool.place([n, 20])
    pool.fill(table, [n, 20])
    lens = [min(n, i + 1) for i in range(tokens)] + [20]
    lse = np.full((tokens + 1, H), 4.0, dtype=np.float32)
    _watch(pool, table, [tokens, 1], lens, H, decay=0.5, lse=lse)


def test_weights_of_fewer_tokens_than_rows():
    # a batch whose last rows have no token in this step: their weights stay
    pool = Pool(60, 16, 16, seed=92)
    full = [100, 33, 50, 7]
    table = pool.place(full)
    pool.fill(table, full)
    smla = _smla()
    rng = np.random.default_rng(93)
    q = bf16(rng.standard_normal((2, 32, 512)))
    lse = _lse(q, pool, table, [0, 1, 2, 2, 2], full[:2])
    out = _f32(np.full((4, table.shape[1] * 16), 3.0))
    smla.cache_weights(bf16_dev(q), pool.device(), _i32(table), _i32(full[:2]), _f32(lse), out)
    ref, bound = M.weights(q, pool.codes, pool.scales, table, [0, 1, 2, 2, 2], full[:2], lse, np.full(out.shape, 3.0), 1.0,
                           np.full(out.shape, 3.0, dtype=np.float32), 16, 16)
    got = out.double().cpu().numpy()
    assert (np.abs(got - ref) <= bound).all() and (got[2:] == 3.0).all()


def test_decode_calls_refuse_what_they_cannot_take():
    smla = _smla()
    from sparse_mla_attention_gb300 import SmlaError, _lib
    pool = Pool(20, 16, 16, seed=94)
    table = pool.place([40, 20], extra=0)
    cache = pool.device()
    tt, lt = _i32(table), _i32([40, 20])
    W = table.shape[1] * 16
    w, q, lse = torch.zeros((2, W), device=DEV), bf16_dev(np.zeros((2, 16, 512))), torch.zeros((2, 16), device=DEV)
    weights = lambda **k: smla.cache_weights(**{**dict(q=q, cache=cache, table=tt, lens=lt, lse=lse, weights=w), **k})
    evict = lambda **k: smla.cache_evict(**{**dict(cache=cache, table=tt, lens=lt, weights=w, keep=8), **k})
    reorder = lambda **k: smla.cache_reorder(**{**dict(cache=cache, table=tt, lens=lt, parents=_i32([0, 1])), **k})
    for call, kind, bad in ((weights, ValueError, dict(lens=_i32([1]))), (weights, ValueError, dict(lse=lse[:, :8])),
                            (weights, ValueError, dict(weights=torch.zeros((2, W + 16), device=DEV))),
                            (weights, TypeError, dict(weights=w.double())), (weights, ValueError, dict(earlier=w[:1])),
                            (weights, ValueError, dict(cu_tokens=_i32([0, 2]))), (weights, ValueError, dict(table=tt[:1])),
                            (weights, ValueError, dict(q=q.transpose(0, 1))), (weights, TypeError, dict(lens=lt.long())),
                            (evict, ValueError, dict(keep=0)), (evict, ValueError, dict(keep=W + 1)),
                            (evict, ValueError, dict(first=5, recent=4)), (evict, ValueError, dict(first=-1)),
                            (evict, ValueError, dict(weights=w.t())), (evict, ValueError, dict(lens=lt.cpu())),
                            (evict, ValueError, dict(out=(tt.clone(), lt.clone(), w.clone(), _i32(np.zeros((2, 9)))))),
                            (reorder, TypeError, dict(parents=torch.zeros(2, device=DEV))),
                            (reorder, ValueError, dict(weights=w[:1])),
                            (reorder, ValueError, dict(out=(tt.clone(), lt.clone(), w.clone())))):
        with pytest.raises(kind):
            call(**bad)
    for call, bad, code in ((weights, dict(decay=float("nan")), _lib.SMLA_ERR_ARG),
                            (weights, dict(scale=-1.0), _lib.SMLA_ERR_ARG),
                            (evict, dict(out=(tt, lt.clone(), w.clone(), _i32(np.zeros((2, 8))))), _lib.SMLA_ERR_OVERLAP),
                            (reorder, dict(out=(tt, lt.clone(), None)), _lib.SMLA_ERR_OVERLAP)):
        with pytest.raises(SmlaError) as e:
            call(**bad)
        assert e.value.code == code
    x, s = torch.zeros((6, 50), device=DEV), torch.zeros((2, 3), device=DEV)
    for kind, args, kw in ((TypeError, (x.double(), s), {}), (ValueError, (x[:5], s), {}), (ValueError, (x.t(), s), {}),
                           (ValueError, (x, s), dict(done=torch.zeros((2, 3), dtype=torch.bool, device=DEV))),
                           (TypeError, (x, s), dict(done=torch.zeros((2, 3), device=DEV), eos=1)),
                           (SmlaError, (x, s), dict(out=(tt, tt, tt.float()))),         # (of the right shape, but one tensor twice)
                           (ValueError, (x, s), dict(n=2, out=(tt, tt, tt.float()))), (SmlaError, (x, s), dict(n=65)),
                           (SmlaError, (x, s), dict(n=0)), (ValueError, (x.cpu(), s), {})):
        with pytest.raises(kind):
            smla.beam_select(*args, **kw)
    pool.check(cache)


@pytest.mark.parametrize("page", [16, 256])
def test_what_is_kept_is_attended_to_as_before(page):
    # attention over the kept rows is attention over the picks of the same positions
    smla = _smla()
    rng = np.random.default_rng(95)
    lens = [700, 300, 90]
    pool = Pool(300, page, 16, seed=96)
    table = pool.place(lens)
    pool.fill(table, lens)
    cache = pool.device()
    tt, lt = _i32(table), _i32(lens)
    q = bf16_dev(rng.standard_normal((3, 48, 512)))
    o, lse = smla.sparse_mla_fwd_paged(q, cache, tt, lt)
    w = smla.cache_weights(q, cache, tt, lt, lse, torch.zeros((3, table.shape[1] * page), device=DEV))
    # a head's weights sum to 1 (lse and each weight off by a few 2^-20)
    np.testing.assert_allclose(w.double().sum(1).cpu().numpy(), 48.0, rtol=1e-4)
    new, new_lens, _, kept = smla.cache_evict(cache, tt, lt, w, 128, first=4, recent=16)
    a, la = smla.sparse_mla_fwd_paged(q, cache, new, new_lens)
    b, lb = smla.sparse_mla_fwd_paged(q, cache, tt, lt, topk=kept)
    pool.refcount[:] = _np(cache.refcount)
    ref, rl, ob, lbound = R.attend(to_f64(q), pool.codes, pool.scales, table, lens, page, 16, topk=_np(kept))
    for got, gl in ((a, la), (b, lb)):                 # (scales may have grown: codes rounded to 2^-4 of the values at most)
        assert (np.abs(gl.double().cpu().numpy() - rl) <= lbound + 2.0 ** -4).all()
    assert (np.abs(to_f64(b) - ref) <= ob).all()
    err = np.linalg.norm(to_f64(a) - ref) / np.linalg.norm(ref)
    assert err <= 2.0 ** -4
