"""Prefix groups from a slot table against the definition, over many small random tables and a few wide ones."""

import numpy as np
import pytest

import radixattention_prefix_shared_radix_gb300 as sgl
from oracle.groups import prefix_groups, prefix_groups_bruteforce


def _groups(table, lens):
    g = sgl.sgl_groups_create()
    try:
        sgl.sgl_groups_from_table(table, lens, g)
        return sgl.groups_as_numpy(sgl.sgl_groups_view(g))
    finally:
        sgl.sgl_groups_destroy(g)


def _same(a, b):
    for k in b:
        assert np.array_equal(np.asarray(a[k]), np.asarray(b[k])), k


@pytest.mark.parametrize("seed", range(4))
def test_small_tables(seed):
    """Few distinct slots, so that rows share, end inside, equal and prefix one another in every way."""
    rng = np.random.default_rng(seed)
    for i in range(400):
        B, ld, k = int(rng.integers(0, 9)), int(rng.integers(1, 9)), int(rng.integers(1, 4))
        table = rng.integers(-1, k, (B, ld)).astype(np.int32)
        lens = rng.integers(0, ld + 1, B).astype(np.int32)
        if i % 3 == 0 and B:
            table[rng.integers(0, B)] = table[0]
        _same(_groups(table, lens), prefix_groups_bruteforce([table[r, :lens[r]] for r in range(B)]))


@pytest.mark.parametrize("B,shared,own", [(1, 0, 700), (64, 300, 40), (200, 64, 3), (17, 0, 900)])
def test_wide_tables(B, shared, own):
    rng = np.random.default_rng(B)
    table = rng.permutation(B * (shared + own) + 1)[:B * (shared + own)].reshape(B, -1).astype(np.int32)
    table[:, :shared] = table[0, :shared]
    table[B // 2:, :shared // 2] = rng.permutation(10 ** 6)[:shared // 2]
    lens = rng.integers(0, shared + own + 1, B).astype(np.int32)
    _same(_groups(table, lens), prefix_groups(table, lens))
