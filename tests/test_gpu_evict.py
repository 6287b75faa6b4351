"""Eviction by scores on the GPU against the oracle: which tokens stay is whole numbers, held to equality."""

import numpy as np
import pytest
import torch

import radixattention_prefix_shared_radix_gb300 as sgl
from oracle import evict as oevict

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from radixattention_prefix_shared_radix_gb300 import build
    build.build()


def _scores(kind, shape, rng):
    if kind == "spread":
        return np.exp(2 * rng.standard_normal(shape)).astype(np.float32)
    if kind == "ties":
        return rng.integers(0, 4, shape).astype(np.float32)
    if kind == "equal":
        return np.full(shape, 0.25, dtype=np.float32)
    if kind == "close":       # the last of the bits that tell them apart
        return (np.float32(1.0) + rng.integers(0, 300, shape) * np.float32(2.0 ** -23)).astype(np.float32)
    x = rng.standard_normal(shape).astype(np.float32)
    odd = np.array([np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-45, -1e-45, 3.4028235e38, -3.4028235e38], dtype=np.float32)
    at = rng.random(shape) < 0.5
    x[at] = odd[rng.integers(0, len(odd), int(at.sum()))]
    return x


class Rows:
    def __init__(self, lens, budgets, scores, ld=None, sld=None, seed=0):
        self.rng = np.random.default_rng(seed)
        self.lens, self.budgets = np.array(lens, dtype=np.int32), np.array(budgets, dtype=np.int32)
        self.B = len(lens)
        most = max(int(self.lens.max()), 1)
        self.ld, self.sld = ld or most, sld or most
        self.scores = _scores(scores, (self.B, self.sld), self.rng)
        self.table = self.rng.integers(-5, 2 ** 31 - 1, (self.B, self.ld)).astype(np.int32)
        self.pos = np.cumsum(self.rng.integers(1, 4, (self.B, self.ld)), 1).astype(np.int32)

    def run(self, page=1, sinks=0, recent=0, in_place=False, positions=True, evicted=True, eld=None, stream=None):
        d = [torch.from_numpy(x).cuda() for x in (self.scores, self.table, self.pos, self.lens)]
        out = d if in_place else [torch.full_like(x, 77) for x in d]
        bud = torch.from_numpy(self.budgets).cuda()
        ev = torch.full((self.B, self.ld if eld is None else eld), 99, dtype=torch.int32, device="cuda") if evicted else None
        cnt = torch.full((self.B,), 99, dtype=torch.int32, device="cuda")
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        sgl.sgl_kv_evict(d[0], d[1], d[3], bud, out[0], out[1], out[3], ws, ev, cnt, d[2] if positions else None,
                         out[2] if positions else None, page, sinks, recent, stream)
        torch.cuda.synchronize()
        return [x.cpu().numpy() for x in out], None if ev is None else ev.cpu().numpy(), cnt.cpu().numpy(), ws

    def check(self, page=1, sinks=0, recent=0, in_place=False, positions=True, **kw):
        (s, t, p, n), ev, cnt, ws = self.run(page, sinks, recent, in_place, positions, **kw)
        sgl.sgl_check(ws)
        same = lambda a, b: np.array_equal(a, b, equal_nan=a.dtype == np.float32)   # noqa: E731
        for r in range(self.B):
            L = int(self.lens[r])
            stays = oevict.keep(self.scores[r, :L], int(self.budgets[r]), page, sinks, recent)
            m = int(stays.sum())
            assert n[r] == m and cnt[r] == L - m, (r, L, m, n[r], cnt[r])
            for got, was, fill in ((s, self.scores, 0), (t, self.table, -1)) + (((p, self.pos, -1),) if positions else ()):
                assert same(got[r, :m], was[r, :L][stays]), (r, L, m)
                assert (got[r, m:L] == fill).all()
                # past the row's end: as it was
                rest = was[r, L:] if in_place else np.full_like(was[r, L:], 77)
                assert same(got[r, L:], rest)
            if ev is not None:
                assert np.array_equal(ev[r, :L - m], self.table[r, :L][~stays])
                assert (ev[r, L - m:] == 99).all()


KINDS = ["spread", "ties", "equal", "close", "odd"]


@pytest.mark.parametrize("scores", KINDS)
@pytest.mark.parametrize("page", [1, 16, 5])
@pytest.mark.parametrize("in_place", [False, True])
def test_short_rows(scores, page, in_place):
    lens = [0, 1, 2, 15, 16, 17, 31, 33, 64, 100, 129, 500, 500, 500, 500, 500]
    budgets = [0, 0, 1, 7, 16, 16, 1000, 20, -5, 3, 128, 499, 500, 1, 250, 0]
    r = Rows(lens, budgets, scores, ld=600, sld=520)
    for sinks, recent in ((0, 0), (4, 32), (1, 1), (600, 3), (0, 700), (17, 0)):
        r.check(page, sinks, recent, in_place)


@pytest.mark.parametrize("n", [8191, 8192, 8193, 16384, 16385, 40000, 131072, 140001])
@pytest.mark.parametrize("page,sinks,recent", [(1, 4, 64), (16, 16, 100), (7, 0, 0)])
@pytest.mark.parametrize("in_place", [False, True])
def test_long_rows(n, page, sinks, recent, in_place):
    """Both sides of the sizes at which more CTAs take a row, and rows of several rounds of moves."""
    for scores in ("spread", "ties"):
        lens = [n, n // 2, n - 1, 10, 0]
        r = Rows(lens, [n // 3, 64, n - 2, 5, 0], scores, seed=n)
        r.check(page, sinks, recent, in_place, positions=scores == "ties")


@pytest.mark.parametrize("page", [32, 64, 100, 999, 2048, 2 ** 28, 2 ** 30 - 1])
@pytest.mark.parametrize("in_place", [False, True])
def test_pages_as_long_as_rows_and_longer(page, in_place):
    lens = [0, 1, 31, 32, 33, 64, 99, 100, 101, 999, 1000, 2000, 2048, 9000]
    r = Rows(lens, [n // 2 for n in lens], "spread", seed=3)
    for sinks, recent in ((0, 0), (40, 10)):
        r.check(page, sinks, recent, in_place)
    r = Rows(lens[:-1], [n // 3 for n in lens[:-1]], "ties", seed=4)
    r.check(page, 0, 5, in_place)


def test_empty_tables_and_batches():
    f, t = torch.zeros(2, 0, device="cuda"), torch.zeros(2, 0, dtype=torch.int32, device="cuda")
    n = torch.zeros(2, dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    sgl.sgl_kv_evict(f, t, n, n, f, t, torch.full_like(n, 5), ws)
    sgl.sgl_check(ws)
    e = n[:0]
    sgl.sgl_kv_evict(f[:0], t[:0], e, e, f[:0], t[:0], e, ws)
    sgl.sgl_check(ws)


def test_the_longest_rows():
    """786432 pages are the most."""
    n = 786432
    r = Rows([n, n - 3], [n // 2, 1000], "ties", seed=1)
    r.check(1, 4, 100, True)
    too = torch.zeros(1, n + 1, device="cuda")
    t = torch.zeros(1, n + 1, dtype=torch.int32, device="cuda")
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    with pytest.raises(sgl.SglError) as e:
        sgl.sgl_kv_evict(too, t, one, one, too, t, one, ws)
    assert e.value.status == -3
    sgl.sgl_kv_evict(too, t, one, one, too, t, one, ws, page_size=2)
    sgl.sgl_check(ws)


def test_many_requests():
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 700, 400)
    Rows(lens, rng.integers(0, 700, 400), "spread").check(1, 2, 16, True)
    Rows(lens, rng.integers(0, 700, 400), "spread").check(16, 2, 16, False, evicted=False)


def test_bad_lengths_and_short_lists_are_reported():
    r = Rows([40, 30, 20], [10, 10, 10], "spread", ld=40)
    good = r.run()
    r.lens[0], r.lens[1] = 41, -3                 # beyond the row; negative: as the nearest end
    (s, t, p, n), ev, cnt, ws = r.run()
    with pytest.raises(sgl.SglError) as e:
        sgl.sgl_check(ws)
    assert e.value.status == -5
    assert n.tolist() == [10, 0, 10] and cnt.tolist() == [30, 0, 10]
    assert np.array_equal(t[0, :40], good[0][1][0, :40]) and (t[1] == 77).all()
    sgl.sgl_check(ws)
    r = Rows([40, 30], [10, 25], "spread")
    (s, t, p, n), ev, cnt, ws = r.run(eld=7)
    with pytest.raises(sgl.SglError):
        sgl.sgl_check(ws)
    assert cnt.tolist() == [30, 5]
    gone = r.table[0][~oevict.keep(r.scores[0], 10)]
    assert np.array_equal(ev[0], gone[:7]) and (ev[1, 5:] == 99).all()


def test_in_a_graph_and_on_another_stream():
    """A captured eviction in place, replayed as a loop does: a token is added, one leaves."""
    B, ld, budget, recent = 5, 300, 200, 8
    rng = np.random.default_rng(9)
    scores = torch.from_numpy(_scores("spread", (B, ld), rng)).cuda()
    table = torch.arange(B * ld, dtype=torch.int32, device="cuda").view(B, ld)
    pos = torch.arange(ld, dtype=torch.int32, device="cuda").repeat(B, 1)
    lens = torch.tensor([200, 250, 3, 0, 200], dtype=torch.int32, device="cuda")
    bud = torch.full((B,), budget, dtype=torch.int32, device="cuda")
    ev, cnt = torch.zeros(B, ld, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            sgl.sgl_kv_evict(scores, table, lens, bud, scores, table, lens, ws, ev, cnt, pos, pos, recent=recent)
    h = [x.cpu().numpy().copy() for x in (scores, table, pos, lens)]
    for step in range(4):
        for r in range(B):                        # a new token at each row's end
            n = int(h[3][r])
            h[0][r, n], h[1][r, n], h[2][r, n] = 0.5 * step, 5000 + 10 * step + r, 1000 + step
            h[3][r] += 1
        for x, y in zip((scores, table, pos, lens), h):
            x.copy_(torch.from_numpy(y))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for r in range(B):
            n = int(h[3][r])
            stays = oevict.keep(h[0][r, :n], budget, recent=recent)
            m = int(stays.sum())
            for y, fill in ((h[0], 0), (h[1], -1), (h[2], -1)):
                y[r, :m], y[r, m:n] = y[r, :n][stays], fill
            h[3][r] = m
        for x, y in zip((scores, table, pos, lens), h):
            assert np.array_equal(x.cpu().numpy(), y)
    sgl.sgl_check(ws)
    r = Rows([700, 900], [100, 200], "spread")
    s2 = torch.cuda.Stream()
    r.check(1, 0, 4, False, stream=s2)


def test_python_arguments_are_checked():
    f = torch.zeros(3, 8, device="cuda")
    t = torch.zeros(3, 8, dtype=torch.int32, device="cuda")
    n = torch.zeros(3, dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    good = dict(scores=f, req_to_token=t, lens=n, budgets=n, scores_out=f, table_out=t, lens_out=n, workspace=ws)
    for bad in (dict(scores=f.double()), dict(req_to_token=t.long()), dict(lens=n.cpu()), dict(budgets=n[:2]),
                dict(scores_out=f[:, :4]), dict(table_out=t[:2]), dict(positions=t), dict(positions=t, positions_out=t[:2]),
                dict(evicted=t[:2]), dict(evicted_count=n[:1]), dict(scores=f[:2])):
        with pytest.raises((TypeError, ValueError)):
            sgl.sgl_kv_evict(**dict(good, **bad))
    for bad in (dict(page_size=0), dict(sinks=-1), dict(recent=-1), dict(workspace=ws[:128])):
        with pytest.raises(sgl.SglError):
            sgl.sgl_kv_evict(**dict(good, **bad))
    sgl.sgl_kv_evict(**good)
    sgl.sgl_check(ws)
