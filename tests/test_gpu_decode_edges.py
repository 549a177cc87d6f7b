"""GPU tests of the decode calls (accumulated weights, eviction, beam selection, reordering) where they can go wrong:
sequences without a choice in wide tables, equal candidates in rows of every alignment, pages that nobody owns, odd scales
and page numbers."""

import numpy as np
import pytest
import torch

import decode_reference as M
from test_gpu_cache import DEV, Pool, _i32, _smla, bf16, bf16_dev
from test_gpu_decode import _evict_and_check, _f32, _heavy, _lse, _np, _watch

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------------------ eviction
@pytest.mark.parametrize("lens,keep,first,recent", [
    ([20000, 0, 1, 500], 500, 0, 0), ([20000, 0, 1, 500], 500, 200, 300), ([20000, 16385, 17000], 1, 0, 1),
    ([20000, 16385, 17000], 1, 1, 0), ([0] * 40 + [20000] + [0] * 40, 20000, 5, 5), ([0, 0, 0, 30000, 2], 25000, 0, 25000)])
def test_evict_of_sequences_without_a_choice_in_wide_tables(lens, keep, first, recent):
    rng = np.random.default_rng(keep)
    pool = Pool(1200, 64, 64, seed=100, junk=False)
    table = pool.place(lens)
    assert table.shape[1] * 64 > 16384
    _evict_and_check(pool, table, lens, _heavy(rng, len(lens), table.shape[1] * 64), keep, first, recent)


# ------------------------------------------------------------------------------------------------ beams
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def _picked(x, scores, n):
    got = _smla().beam_select(x, _f32(scores), n=n)
    return _np(got[0]), _np(got[1]), got[2].double().cpu().numpy()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V,pad", [(1, 0), (3, 0), (7, 0), (9, 0), (17, 0), (31, 2), (9001, 0), (9000, 1), (9000, 3), (16385, 0),
                                   (32001, 0), (32767, 0), (32769, 0), (50001, 0), (50257, 5), (65537, 0), (151665, 0)])
def test_equal_beams_in_rows_of_any_alignment(dtype, V, pad):
    # equal rows have equal log-sums wherever they start: of equal candidates the lower beam's comes first
    g = torch.Generator(device=DEV).manual_seed(V)
    one = torch.randn(3, 1, V, generator=g, device=DEV) * 3
    x = torch.full((24, V + pad), 50.0, device=DEV)
    x[:, :V] = one.expand(3, 8, V).reshape(24, V)
    x = x.to(dtype)[:, :V]
    scores = np.repeat(-np.arange(3.0)[:, None], 8, 1)
    for n in (8, 20):
        p, t, s = _picked(x, scores, n)
        ref = M.select(x.double().cpu().numpy(), scores, n)
        np.testing.assert_array_equal(p, ref[0])
        np.testing.assert_array_equal(t, ref[1])
        for b in range(3):                             # a token's scores are the same number
            for v in set(t[b].tolist()):
                assert len(set(s[b][t[b] == v].tolist())) == 1


@pytest.mark.parametrize("K,V", [(64, 151936), (60, 200001), (3, 4194304)])
def test_equal_beams_of_more_chunks_than_a_part(K, V):
    g = torch.Generator(device=DEV).manual_seed(K)
    x = (torch.randn(1, V, generator=g, device=DEV) * 3).expand(K, V).contiguous()
    p, t, _ = _picked(x, np.zeros((1, K)), 64)
    best = torch.sort(x[0], descending=True, stable=True)[1][:64].tolist()
    want = [(k, v) for v in best for k in range(K)][:64]
    assert list(zip(p[0].tolist(), t[0].tolist())) == want


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("before", [-1e9, -1e20, 1e20, float(np.finfo(np.float32).min)])
def test_beams_of_huge_scores_go_by_their_logits(dtype, before):
    # in 64 bits such a beam's scores are equal or nearly so: what its logits say still holds
    g = torch.Generator(device=DEV).manual_seed(7)
    x = (torch.randn(4, 40001, generator=g, device=DEV)).to(dtype)
    x[3] = x[2]
    scores = np.array([[before] * 2, [before * 2 if abs(before) < 1e30 else before, before]])
    n = 12
    p, t, _ = _picked(x, scores, n)
    v = x.double().cpu().numpy()
    for b in range(2):
        s = scores[b].astype(np.float32).astype(np.float64)
        lse = [np.log(np.exp(v[2 * b + k]).sum()) for k in range(2)]
        cand = []
        for k in range(2):
            order = np.lexsort((np.arange(v.shape[1]), -v[2 * b + k]))[:n]
            cand += [(-(s[k] + (v[2 * b + k, i] - lse[k])), k, -v[2 * b + k, i], i) for i in order]
        if before == -1e9:                             # (scores apart by less than the log-sums' own error are not held apart)
            got = [(a, c) for a, c in zip(p[b], t[b])]
            for k in range(2):
                mine = [c for a, c in got if a == 2 * b + k]
                order = np.lexsort((np.arange(v.shape[1]), -v[2 * b + k]))
                assert mine == order[:len(mine)].tolist()
        else:
            want = [(2 * b + k, i) for _, k, _, i in sorted(cand)[:n]]
            assert list(zip(p[b].tolist(), t[b].tolist())) == want


# ------------------------------------------------------------------------------------------------ weights
@pytest.mark.parametrize("counts", [[1, 1, 1], [40, 1, 40]])           # few rows of q a sequence, and many
def test_weights_report_every_page_out_of_range_and_take_any_scale(counts):
    from sparse_mla_attention_gb300 import SmlaError, _lib
    smla = _smla()
    rng = np.random.default_rng(10)
    pool = Pool(60, 16, 16, seed=11)
    full = [300, 45, 130]
    table = pool.place(full)
    pool.fill(table, full)
    cu = np.concatenate([[0], np.cumsum(counts)])
    lens = [n - c + 1 + i for n, c in zip(full, counts) for i in range(c)]
    T, W = len(lens), table.shape[1] * 16
    q = bf16(rng.standard_normal((T, 32, 512)))
    lse = _lse(q, pool, table, cu, lens)
    zero = np.zeros((3, W), dtype=np.float32)
    ref, bound = M.weights(q, pool.codes, pool.scales, table, cu, lens, lse, zero, 0.0, zero, 16, 16)
    args = lambda t: (bf16_dev(q), pool.device(), _i32(t), _i32(lens), _f32(lse))
    for page in (-1, 60, 1 << 30, -(1 << 31), (1 << 31) - 1):
        for b, j in ((0, 0), (0, 17), (2, 8)):
            bad = table.astype(np.int64).copy()
            bad[b, j] = page
            out = torch.zeros((3, W), device=DEV)
            with pytest.raises(SmlaError) as e:
                smla.cache_weights(*args(bad), out, cu_tokens=_i32(cu))
            assert e.value.code == _lib.SMLA_ERR_INDEX
            live = np.ones((3, W), dtype=bool)
            live[b, 16 * j:16 * j + 16] = False
            got = out.double().cpu().numpy()
            assert (np.abs(got - ref)[live] <= bound[live]).all() and (got[~live] == 0).all()
    # a block whose scale is not a number says so in its positions; one below zero counts as it is
    for scale in (np.nan, -0.25):
        was, pool.scales[table[0, 3], 0] = pool.scales[table[0, 3], 0], scale
        out = smla.cache_weights(*args(table), torch.zeros((3, W), device=DEV), cu_tokens=_i32(cu)).double().cpu().numpy()
        odd = np.zeros((3, W), dtype=bool)
        odd[0, 48:64] = True
        assert (np.abs(out - ref)[~odd] <= bound[~odd]).all()
        if np.isnan(scale):
            assert np.isnan(out[odd]).all()
        else:
            r, o = M.weights(q, pool.codes, pool.scales, table, cu, lens, lse, zero, 0.0, zero, 16, 16)
            assert (np.abs(out - r)[odd] <= o[odd]).all()
        pool.scales[table[0, 3], 0] = was


# ------------------------------------------------------------------------------------------------ pages that nobody owns
@pytest.mark.parametrize("page,lens,keep", [(16, [100, 80, 33], 60), (64, [20000, 300], 9000)])
def test_evict_refuses_sequences_with_pages_that_nobody_owns(page, lens, keep):
    # such a page is free, and the lowest free ones are what the kept rows would be written to
    from sparse_mla_attention_gb300 import SmlaError, _lib
    smla = _smla()
    rng = np.random.default_rng(3)
    for b, j in ((0, 0), (1, 2), (0, 3)):
        pool = Pool(800, page, 16, seed=110)
        table = pool.place(lens, extra=2)
        pool.fill(table, lens)
        pool.refcount[table[b, j]] = 0
        w = _heavy(rng, len(lens), table.shape[1] * page)
        cache = pool.device()
        out = (_i32(table), _i32(lens), _f32(w), _i32(np.zeros((len(lens), keep))))
        with pytest.raises(SmlaError) as e:
            smla.cache_evict(cache, _i32(table), _i32(lens), _f32(w), keep, out=out)
        assert e.value.code == _lib.SMLA_ERR_REFCOUNT
        assert (out[0] == -1).all() and (out[1] == 0).all()
        pool.check(cache)
    # entries behind a sequence's length are not looked at
    pool = Pool(800, page, 16, seed=111)
    table = pool.place(lens, extra=2)
    pool.fill(table, lens)
    table[:, -1] = np.flatnonzero(pool.refcount == 0)[:len(lens)]
    _evict_and_check(pool, table, lens, _heavy(rng, len(lens), table.shape[1] * page), keep, 1, 2)


@pytest.mark.parametrize("last", [0, 5])                               # the parent ends with its page, or each child copies one
@pytest.mark.parametrize("n", [40, 5000])
def test_reorder_leaves_out_pages_that_nobody_owns(n, last):
    from sparse_mla_attention_gb300 import SmlaError, _lib
    smla = _smla()
    page, full = 16, 6
    lens = [full * page + last, 3 * page, 2 * page]
    pool = Pool(30 + n, page, 16, seed=120, junk=False)
    table = pool.place(lens)
    loose, ended = table[0, 2], table[1, 1]            # one that n - 1 children would share, one of a row that ends
    pool.refcount[[loose, ended]] = 0
    cache = pool.device()
    ws = smla.Workspace(DEV)
    out = (_i32(np.zeros((n + 1, table.shape[1]))), _i32(np.zeros(n + 1)), None)
    with pytest.raises(SmlaError) as e:
        smla.cache_reorder(cache, _i32(table), _i32(lens), _i32([0] * n + [2]), out=out, workspace=ws)
    assert e.value.code == _lib.SMLA_ERR_REFCOUNT
    got, count = _np(out[0]), _np(cache.refcount)
    np.testing.assert_array_equal(got[0], table[0])
    assert (got[1:n, 2] == -1).all()
    own = [j for j in range(full) if j != 2]
    assert (got[1:n][:, own] == table[0][own]).all() and (count[table[0][own]] == n).all()
    free = np.flatnonzero(pool.refcount == 0)[:n - 1 if last else 0]
    if last:
        np.testing.assert_array_equal(got[1:n, full], free)
    want = pool.refcount.copy()
    want[table[0][own]] = n
    want[[table[1, 0], table[1, 2]]] = 0
    want[free] = 1
    np.testing.assert_array_equal(count, want)


# ------------------------------------------------------------------------------------------------ what small parts of the inputs do
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["normal", "flat", "rising", "falling", "peaked"])
def test_selections_scores_are_as_exact_as_their_sums(dtype, kind):
    # A value d below its row's maximum passes up to 13 additions, 8 scalings by an approximate power (2^-22, and 2^-24 for the
    # product), one power of its own, and arguments off by 2.7 d 2^-24 in all (a subtraction, the factor log2(e), the
    # product): relative to the sum 2^-24 (13 + 8 * 5 + 4 + 2.7 sum_i w_i d_i), w_i its softmax. The score's own rounding
    # is 2^-24 of it.
    V = 50001
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randn(6, V, generator=g, device=DEV) * 3
    if kind == "flat":
        x = x * 1e-3
    elif kind in ("rising", "falling"):
        x = torch.sort(x, dim=1, descending=kind == "falling")[0]
    elif kind == "peaked":
        x[:, ::5000] += 20.0
    x = x.to(dtype)
    scores = -np.arange(6.0).reshape(2, 3) / 8
    p, t, s = _picked(x, scores, 9)
    v = x.double().cpu().numpy()
    ref = M.select(v, scores, 9)
    np.testing.assert_array_equal(p, ref[0])
    np.testing.assert_array_equal(t, ref[1])
    top = v.max(axis=1, keepdims=True)
    w = np.exp(v - top)
    d = (w * (top - v)).sum(axis=1) / w.sum(axis=1)
    bound = 2.0 ** -24 * (np.abs(ref[2]) + 57 + 2.7 * d[p])
    assert (np.abs(s - ref[2]) <= bound).all()


@pytest.mark.parametrize("tokens", [1, 40])                            # both forms
def test_weights_see_every_bit_of_q(tokens):
    # One value a cached row, 448 in column p % 512: a score is one product of q, exact in fp32 (8 x 4 bits) where q's two parts
    # hold it, which is for 2^-13 of the row's largest (here 1) and more; below that they are off by up to 2^-21 of it.
    # The argument: factors scale, log2(e) and their product, lse in log2 units, the sum; the power 2^-22; up to 16 * tokens
    # additions a position (16 columns at a time as a tree, so fewer).
    smla = _smla()
    rng = np.random.default_rng(130)
    H, L, page = 16, 1024, 64
    pool = Pool(40, page, 64, seed=131, junk=False)
    table = pool.place([L])
    pool.codes[:] = 0
    pool.scales[:] = 1.0
    for p in range(L):
        pool.codes[table[0, p // page], p % page, p % 512] = 0x7E
    q = np.exp2(rng.uniform(-18, 0, size=(tokens, H, 512))) * rng.choice([-1.0, 1.0], size=(tokens, H, 512))
    q[:, :, 0] = 1.0
    q = np.clip(bf16(q), -1.0, 1.0)
    lse = rng.uniform(1, 5, size=(tokens, H)).astype(np.float32)
    W = table.shape[1] * page
    out = smla.cache_weights(bf16_dev(q), pool.device(), _i32(table), _i32([L] * tokens), _f32(lse),
                             torch.zeros((1, W), device=DEV), cu_tokens=_i32([0, tokens]))
    got = out.double().cpu().numpy()[0, :L]
    a = q[:, :, np.arange(L) % 512] * 448.0 / np.sqrt(512.0)
    l = lse[:, :, None].astype(np.float64)
    w = np.exp(a - l)
    d = 2.0 ** -24 * (5 * np.abs(a) + 3 * l + 2 * np.abs(a - l) + 16 * tokens + 4) + 2.0 ** -22
    d = d + np.where(np.abs(q) < 2.0 ** -13, 2.0 ** -21, 0.0)[:, :, np.arange(L) % 512] * 448.0 / np.sqrt(512.0)
    assert (np.abs(got - w.sum(axis=(0, 1))) <= (w * np.expm1(d)).sum(axis=(0, 1))).all()


@pytest.mark.parametrize("most", [3, 40])                              # few rows of q a sequence, and many
def test_weights_of_more_sequences_than_a_block_has_threads(most):
    rng = np.random.default_rng(140)
    B = 1100
    full = rng.integers(0, 150, size=B)
    full[5], full[1099] = 2000, 700
    counts = [int(min(n, c)) for n, c in zip(full, rng.integers(0, most + 1, size=B) * (rng.random(B) < 0.5))]
    counts[5], counts[7] = 2 * most, 0
    pool = Pool(12000, 16, 16, seed=141, junk=False)
    table = pool.place(full)
    pool.fill(table, full)
    lens = [n - c + 1 + i for n, c in zip(full, counts) for i in range(c)]
    _watch(pool, table, counts, lens, 16 if most == 3 else 48, decay=0.5, lse=np.full((len(lens), 16 if most == 3 else 48), 3.0, np.float32))
