"""Pins of the oracle's 4-bit format and rotation (no GPU)."""

import numpy as np
import pytest

from oracle import fp4, rope


def test_e2m1_codes_are_the_nearest_values():
    assert np.array_equal(fp4.float_to_e2m1(fp4.e2m1_to_float(np.arange(16))), np.arange(16))
    # ties go to the even code; beyond 6 saturates
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    assert list(fp4.e2m1_to_float(fp4.float_to_e2m1(ties))) == [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0]
    assert list(fp4.e2m1_to_float(fp4.float_to_e2m1([5.01, 7.0, -100.0, np.inf]))) == [6.0, 6.0, -6.0, 6.0]


def test_quantised_blocks_stay_within_half_a_step():
    x = np.random.default_rng(1).standard_normal((50, 3, 64)).astype(np.float32)
    codes, sf = fp4.quantise(x, 0.75)
    y = fp4.values(fp4.pack(codes, sf), 3, 64, 0.75)
    s = np.repeat(fp4.e4m3_to_float(sf), 16, -1) * 0.75
    # half a step is at most sf (between 4 and 6); the largest value may lie
    # 1/16 of itself above 6 sf, because sf itself was rounded (by 2^-4 at most)
    assert np.all(np.abs(y - x) <= s * (1 + 1e-6))
    # blocks of zeros and of values too small for a scale
    codes, sf = fp4.quantise(np.array([[[0.0] * 16 + [1e-6] * 16]]), 1.0)
    assert not sf.any() and not (codes & 7).any()
    # a NaN marks its block, an infinity saturates
    bad = np.ones((1, 1, 32), dtype=np.float32)
    bad[0, 0, 3], bad[0, 0, 20] = np.nan, np.inf
    codes, sf = fp4.quantise(bad, 1.0)
    assert sf[0, 0, 0] == 0x7F and sf[0, 0, 1] == 0x7E
    assert fp4.e2m1_to_float(codes)[0, 0, 20] == 6.0


@pytest.mark.parametrize("heads,d", [(1, 64), (2, 128), (4, 64), (5, 64), (8, 128), (9, 128)])
def test_pack_and_unpack_are_inverse(heads, d):
    rng = np.random.default_rng(heads * d)
    codes = rng.integers(0, 16, (7, heads, d)).astype(np.uint8)
    sf = rng.integers(0, 256, (7, heads, d // 16)).astype(np.uint8)
    rows = fp4.pack(codes, sf)
    assert rows.shape[1] == fp4.row_bytes(heads, d) and rows.shape[1] % 16 == 0
    c, s = fp4.unpack(rows, heads, d)
    assert np.array_equal(c, codes) and np.array_equal(s, sf)


def test_rotation_keeps_lengths_and_relative_positions():
    rng = np.random.default_rng(2)
    q, k = rng.standard_normal((2, 1, 1, 64))
    for kw in ({}, {"scaling": "yarn", "factor": 4.0, "original": 4096, "low": 1.0, "high": 32.0},
               {"scaling": "banded", "factor": 8.0, "original": 4096, "low": 1.0, "high": 4.0}):
        f = rope.frequencies(64, **kw)
        for pairs in (False, True):
            at = lambda x, p: rope.rotate(x, [p], f, pairs=pairs)[0, 0]  # noqa: E731
            assert np.isclose(np.linalg.norm(at(q, 77)), np.linalg.norm(q))
            assert np.isclose(at(q, 105) @ at(k, 100), at(q, 5) @ at(k, 0))
    assert np.allclose(rope.frequencies(64, scaling="linear", factor=4.0), rope.frequencies(64) / 4)
    # the changed base stretches the slowest pair by the factor and keeps the fastest
    f, g = rope.frequencies(64), rope.frequencies(64, scaling="ntk", factor=8.0)
    assert np.isclose(g[0], f[0]) and np.isclose(g[-1], f[-1] / 8)
