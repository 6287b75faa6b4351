"""Query rows at a log-sum-exp of -infinity add no weight, whatever their elements, the keys and so the products are."""

import numpy as np
import pytest
import torch

import radixattention_prefix_shared_radix_gb300 as sgl
from oracle import fp4
from tests.test_gpu_attn_weights import KINDS, Cache, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from radixattention_prefix_shared_radix_gb300 import build
    build.build()


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (32, 4, 128), (5, 5, 128)])
@pytest.mark.parametrize("decode", [False, True])
def test_queries_of_excluded_rows(kind, bad, hq, hkv, d, decode):
    """Against the same call with zeros in their place: the same bits, and nothing to report."""
    pre, ext = np.array([300, 20, 9]), np.array([1, 1, 1]) if decode else np.array([200, 3, 70])
    c = Cache(kind, pre + ext, hq, hkv, d, seed=d)
    q = c.queries(int(ext.sum()))
    lse = c.lse(q, pre, ext, d ** -0.5)
    first = np.cumsum(ext) - ext
    out = [(first[0], 0), (first[0], hq - 1), (first[2], 1)] if decode else \
        [(0, 0), (17, 1), (18, hq - 1), (199, 2), (200, 0), (202, 3), (203, 0), (272, hq - 1), (250, slice(None))]
    x = q.clone()
    for i, h in out:
        lse[i, h] = -np.inf
        q[i, h] = 0
        x[i, h] = bad
    want = _run(c, q, lse, pre, ext, 0, None, 1.0, decode)
    assert np.isfinite(want).all()
    assert np.array_equal(_run(c, x, lse, pre, ext, 0, None, 1.0, decode), want)
    if not decode:
        for window in (1, 64):
            a, b = (_run(c, y, lse, pre, ext, window, None, 1.0, decode) for y in (q, x))
            assert np.array_equal(a, b)


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("decode", [False, True])
def test_keys_under_excluded_rows(kind, decode):
    """A key of NaN whose token only excluded rows see gets no weight (all rows of request 0; in request 1 other rows do see
    it).  In chunks over other pools than fp32 its own token's score is NaN, and no other."""
    pre, ext = np.array([100, 50]), np.array([1, 1]) if decode else np.array([140, 90])
    c = Cache(kind, pre + ext, 8, 2, 64, seed=2)
    q = c.queries(int(ext.sum()))
    lse = c.lse(q, pre, ext, 0.125)
    lse[:ext[0]] = -np.inf
    clean = _run(c, q, lse, pre, ext, 0, None, 1.0, decode)
    assert not clean[0, :int(pre[0] + ext[0])].any()
    for r, p in ((0, 0), (0, 100), (1, 20)):
        slot = int(c.table[r, p])
        if kind == "fp4":
            codes, sf = fp4.unpack(c.pool.numpy(), 2, 64)
            sf[slot, 1, 2] = 0x7F
            c.pool = torch.from_numpy(fp4.pack(codes, sf))
        elif kind == "fp8":
            c.pool[slot, 1, 33] = 0x7F
        else:
            c.pool[slot, 1, 33] = float("nan")
    got = _run(c, q, lse, pre, ext, 0, None, 1.0, decode)
    assert np.isnan(got[1, 20])
    got[1, 20] = clean[1, 20]
    if not decode and kind != "f32":
        for p in (0, 100):
            assert np.isnan(got[0, p])
            got[0, p] = clean[0, p]
    assert np.array_equal(got, clean)


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("num_sms", [0, 1, 3])
def test_excluded_rows_all_over_long_runs(kind, num_sms):
    """A third of the rows, in runs of up to sixteen query blocks one after the other on few SMs, and blocks of nothing
    else."""
    pre, ext = np.array([700, 0, 33]), np.array([400, 290, 1])
    c = Cache(kind, pre + ext, 16, 2, 64, seed=4)
    q = c.queries(int(ext.sum()))
    lse = 5 + torch.randn(len(q), 16, generator=torch.Generator().manual_seed(5))
    out = torch.rand(len(q), 16, generator=torch.Generator().manual_seed(6)) < 0.3
    out[64:128] = True
    out[690] = True
    lse[out] = -np.inf
    q[out] = 0
    want = _run(c, q, lse, pre, ext, 0, None, 1.0, False, num_sms=num_sms)
    ref, tol = c.expect(q, lse, pre, ext, 0, np.zeros(want.shape, dtype=np.float32), 0.0, False, 0.125)
    live = np.arange(want.shape[1])[None] < (pre + ext)[:, None]
    assert (np.abs(want - ref) <= tol)[live].all() and not want[2, :34].any()
    x = q.clone()
    x[out] = float("nan")
    assert np.array_equal(_run(c, x, lse, pre, ext, 0, None, 1.0, False, num_sms=num_sms), want)
