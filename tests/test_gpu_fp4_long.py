"""Long contexts over a 4-bit cache under one dominant key: weights far below the largest one count in full, however many.

As in tests/test_gpu_fp4.py, but weights enter the second product as f16 values 2^7 times as large, so that each is off by
2^-32 of the largest at most where it is below f16's normal range:
  |O - O64| <= 2^-8 |O64| + (1 + 2^-8) ((2^-11 + 2 delta) A + L 2^-32 max |V|).
"""

import numpy as np
import pytest
import torch

import radixattention_prefix_shared_radix_gb300 as sgl
from oracle import fp4
from tests.test_gpu_fp4 import KS, VS, Batch, _extend, _own, _ref, _star

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from radixattention_prefix_shared_radix_gb300 import build
    build.build()


def _fill(b, first, bits):
    """Keys with a score of `bits` in base 2 at the slot `first` and of zero elsewhere, for queries of ones; values around
    one elsewhere, zero at `first`."""
    hkv, d = b.hkv, b.d
    rng = np.random.default_rng(1)
    k = np.zeros((b.slots, hkv, d), dtype=np.float32)
    k[first] = bits * np.log(2) / np.sqrt(d)          # (sum over d of k / sqrt(d), in base e)
    v = 1 + 0.1 * rng.standard_normal((b.slots, hkv, d)).astype(np.float32)
    v[first] = 0
    b.kp[:], b.vp[:] = fp4.pack(*fp4.quantise(k, KS)), fp4.pack(*fp4.quantise(v, VS))


def _check(b, o, lse, q, r, length):
    slots = b.table[r, :length]
    k, v = fp4.values(b.kp[slots], b.hkv, b.d, KS), fp4.values(b.vp[slots], b.hkv, b.d, VS)
    O, L, to, tl = _ref(q.double().numpy(), k, v, 1 / np.sqrt(b.d))
    wide = (1 + 2.0 ** -8) * length * np.abs(v).max()
    to = to - wide * 2.0 ** -25 + wide * 2.0 ** -32
    err = np.abs(o - O)
    assert (err <= to).all(), "O: worst %.3g of the bound" % (err / to).max()
    assert (np.abs(lse - L) <= tl).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bits", [12.0, 20.0, 24.5, 25.3, 27.0])
def test_extend(d, bits):
    b = Batch(_own([120000]), 8, 1, d, seed=2)
    _fill(b, b.table[0, 11], bits)
    q = torch.ones(2, 8, d, dtype=torch.bfloat16)
    o, lse, *_ = _extend(b, np.array([119998]), np.array([2]), q)
    for i in range(2):
        _check(b, o[i], lse[i], q[i], 0, 119999 + i)


@pytest.mark.parametrize("num_sms", [1, 0])
@pytest.mark.parametrize("bits", [20.0, 25.3])
@pytest.mark.parametrize("shared", [False, True])
def test_decode(num_sms, bits, shared):
    """Pieces as long as the context, when they are planned for one SM; tiles of a shared prefix."""
    b = Batch(_star(20, 60000, 1, 3) if shared else _own([60000]), 8, 1, 128, seed=3)
    _fill(b, b.table[0, 11], bits)
    b.q = torch.ones_like(b.q)
    o, lse = b.run(num_sms=num_sms)
    assert (b.info["num_wide_items"] > 0) == shared
    for r in range(min(b.B, 3)):
        _check(b, o[r], lse[r], b.q[r], r, int(b.lens[r]))
