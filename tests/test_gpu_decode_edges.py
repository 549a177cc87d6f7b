"""GPU tests of the decode calls (accumulated weights, eviction, beam selection, reordering) where they can go wrong:
sequences without a choice in wide tables, equal candidates in rows of every alignment, pages that nobody owns, odd scales
and page numbers."""

import numpy as np
import pytest
import torch

import decode_reference as M
from test_gpu_cache import DEV, Pool, _i32, _smla, bf16, bf16_dev
from test_gpu_decode import _evict_and_check, _f32, _heavy, _lse, _np

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
