"""Attention weights of long chunks against float64 at sampled positions: log-sum-exps are any, so that a position's score
is a sum over the rows that see it and no other position is needed for it."""

import numpy as np
import pytest
import torch

import radixattention_prefix_shared_radix_gb300 as sgl
from tests.test_gpu_attn_weights import Cache, KINDS, _check, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from radixattention_prefix_shared_radix_gb300 import build
    build.build()


def _want(c, q, lse, pre, ext, at, r, adds):
    """float64 scores of request r's positions `at`, and a bound: that of oracle/evict.py for each weight, and `adds`
    additions in sequence."""
    first = int(sum(ext[:r]))
    x, l = q[first:first + ext[r]].cuda(), lse[first:first + ext[r]].cuda().double()
    k = torch.from_numpy(c.keys(r, int(pre[r] + ext[r]))[at]).cuda()
    at = torch.from_numpy(at).cuda()
    seen = at[None] <= int(pre[r]) + torch.arange(int(ext[r]), device="cuda")[:, None]
    sm = c.d ** -0.5
    want, off = (torch.zeros(len(at), dtype=torch.float64, device="cuda") for _ in "ab")
    for h in range(c.hq):
        kh, xh = k[:, h * c.hkv // c.hq], x[:, h].double()
        s = sm * xh @ kh.T - l[:, h, None]
        size = sm * xh.abs() @ kh.abs().T
        w = s.exp().masked_fill_(~seen, 0.0)
        want += w.sum(0)
        off += (w * ((size * (c.d + 12) + s.abs()) * 2.0 ** -24 + 2.0 ** -21)).sum(0)
    return want.cpu().numpy(), (off + want * adds * 2.0 ** -24).cpu().numpy()


@pytest.mark.parametrize("kind,d", [("bf16", 128), ("fp8", 64), ("fp4", 128)])
def test_runs_of_more_than_sixteen_query_blocks(kind, d):
    """64 query heads over 8 KV heads and 27000 tokens: runs of 18 blocks, whose sums a thread adds up in memory.  In
    sequence: 32 columns and 2 of a block, 16 blocks, 2 parts of a run, 94 runs of 8 heads by four threads, 3.  (A run
    that were lost or added twice would be a part in a hundred or more.)"""
    pre, ext = np.array([0, 900]), np.array([27000, 300])
    c = Cache(kind, pre + ext, 64, 8, d, seed=d)
    q = c.queries(int(ext.sum()))
    lse = 6 + torch.randn(len(q), 64, generator=torch.Generator().manual_seed(1))
    got = _run(c, q, lse, pre, ext, 0, None, 1.0, False)
    rng = np.random.default_rng(2)
    for r, n in enumerate(pre + ext):
        edges = np.concatenate([[0, 1, 127, 128, 255, 256, n - 130, n - 129, n - 128, n - 2, n - 1]])
        at = np.unique(np.concatenate([edges, rng.integers(0, n, 80)]))
        want, tol = _want(c, q, lse, pre, ext, at, r, 34 + 16 + 2 + 94 * 2 + 3)
        err = np.abs(got[r, at] - want)
        assert (err <= tol).all(), ((err / tol).max(), at[err > tol][:4])
    assert np.array_equal(_run(c, q, lse, pre, ext, 0, None, 1.0, False), got)     # (in the same order again)


@pytest.mark.parametrize("num_sms,run", [(8, 350), (2, 1398)])
def test_runs_of_hundreds_of_query_blocks(num_sms, run):
    """The same work cut for few SMs: 1688 blocks of 106 tiles and 8 heads, 512 items an SM.  In sequence as above, with
    the parts of a longer run and fewer runs."""
    n = 27000
    c = Cache("fp8", [n], 64, 8, 64, seed=3)
    q = c.queries(n)
    lse = 6 + torch.randn(n, 64, generator=torch.Generator().manual_seed(1))
    assert run == -(-106 * 1688 * 8 // (512 * num_sms))
    got = _run(c, q, lse, np.array([0]), np.array([n]), 0, None, 1.0, False, num_sms=num_sms)
    at = np.unique(np.concatenate([[0, 1, 127, 128, 255, 256, n - 129, n - 1], np.random.default_rng(2).integers(0, n, 80)]))
    want, tol = _want(c, q, lse, [0], [n], at, 0, 34 + 16 + -(-run // 16) + -(-1688 // run) * 2 + 3)
    err = np.abs(got[0, at] - want)
    assert (err <= tol).all(), ((err / tol).max(), at[err > tol][:4])


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("hq,hkv,n", [(2, 2, 11000), (8, 1, 9100), (16, 4, 9473)])
def test_no_item_of_a_long_prompt_is_lost(kind, hq, hkv, n):
    """Log-sum-exps of one size for early and late rows: the last run of query blocks is more than a hundredth of the
    first positions' scores, a full one more, and the bound (weights good to 2^-12, additions in sequence: 34 of a block,
    16 blocks, or 32 weights in fp32, then four threads over the runs of all heads) far below."""
    pre, ext = np.array([0, 700]), np.array([n, 200])
    c = Cache(kind, pre + ext, hq, hkv, 64, seed=n)
    q = c.queries(int(ext.sum()))
    lse = 5 + 0.5 * torch.randn(len(q), hq, generator=torch.Generator().manual_seed(n))
    got = _run(c, q, lse, pre, ext, 0, None, 1.0, False)
    rng = np.random.default_rng(n)
    for r, L in enumerate(pre + ext):
        at = np.unique(np.concatenate([np.arange(4), [127, 128, 255, 256, L - 1], 256 * rng.integers(0, L // 256, 12),
                                       rng.integers(0, L, 60)]))
        runs = -(-int(ext[r]) * hq // hkv // 128 // 4)
        want, tol = _want(c, q, lse, pre, ext, at, r, 34 + 16 + runs * hkv // 4 + 8)
        err = np.abs(got[r, at] - want)
        assert (err <= tol).all(), ((err / tol).max(), at[err > tol][:4])
        assert (tol[at < 4] < 2.0 ** -11 * want[at < 4]).all()


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("num_sms", [1, 5, 400])
def test_work_cut_for_other_numbers_of_sms(kind, num_sms):
    pre, ext = np.array([0, 300, 40]), np.array([290, 70, 0])
    c = Cache(kind, pre + ext, 32, 8, 64, seed=5)
    _check(c, pre, ext, num_sms=num_sms)
    lens = np.array([300, 0, 1, 1000, 65])
    has = (lens > 0).astype(np.int64)
    _check(Cache(kind, lens, 8, 8, 64, seed=6), lens - has, has, decode=True, num_sms=num_sms)


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("lse", [3.3, 5.1, 7.7])
def test_thousands_of_equal_weights(kind, lse):
    """Keys of zeros: 9216 tokens of 8 heads give a position up to 73728 equal weights, whose roundings would all go one
    way in a long chain of additions (4608 in a row: 5e-5 at 5.1).  A weight is off by 2^-24 of its exponent twice and
    by 2^-21; in sequence fp32 pools add 32 weights, 4 lanes and 8 CTAs with three roundings more, the others 34 of a block,
    16 blocks, 36 runs by four threads and 3."""
    n = 9216
    c = Cache(kind, [n], 8, 1, 64, seed=1, spread=0.0)
    q = c.queries(n)
    l = torch.full((n, 8), lse)
    got = _run(c, q, l, np.array([0]), np.array([n]), 0, None, 1.0, False)[0]
    want = 8 * np.arange(n, 0, -1) * np.exp(-np.float64(np.float32(lse)))
    adds = 32 + 4 + 8 + 3 if kind == "f32" else 34 + 16 + 9 + 3
    err = np.abs(got / want - 1)
    assert err.max() <= lse * 2.0 ** -23 + 2.0 ** -21 + adds * 2.0 ** -24, err.max()
