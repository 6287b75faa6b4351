"""Attention weights of cached tokens on the GPU against float64, within the bound that oracle/evict.py derives, and
the run of a loop that thins a cache out: append, attention, weights, eviction."""

import numpy as np
import pytest
import torch

import radixattention_prefix_shared_radix_gb300 as sgl
from oracle import evict as oevict, fp4, rope as orope
from oracle.fp8 import e4m3_to_float
from tests.test_gpu_fp4 import KS, VS

pytestmark = pytest.mark.gpu

KINDS = {"f32": sgl.SGL_DTYPE_F32, "bf16": sgl.SGL_DTYPE_BF16, "fp8": sgl.SGL_DTYPE_BF16_FP8KV,
         "fp4": sgl.SGL_DTYPE_BF16_FP4KV}
HEADS = [(32, 8, 128), (8, 8, 64), (10, 5, 128), (8, 1, 64), (16, 2, 64), (64, 8, 128), (4, 2, 64), (24, 24, 64)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from radixattention_prefix_shared_radix_gb300 import build
    build.build()


class Cache:
    """Requests of `lens` tokens over a paged pool of one kind; slots that no request holds are NaN."""

    def __init__(self, kind, lens, hq, hkv, d, ld=None, page=1, seed=0, spread=1.0):
        self.kind, self.hq, self.hkv, self.d = kind, hq, hkv, d
        self.rng = rng = np.random.default_rng(seed)
        self.lens = np.array(lens, dtype=np.int64)
        self.B, self.ld = len(lens), ld or max(int(max(lens)), 1)
        pages = -(-self.lens // page)
        self.slots = (int(pages.sum()) + 7) * page
        order = rng.permutation(self.slots // page)
        self.table = np.full((self.B, self.ld), -1, dtype=np.int32)
        at = 0
        for r, n in enumerate(self.lens):
            self.table[r, :n] = (order[at:at + pages[r], None] * page + np.arange(page)).reshape(-1)[:n]
            at += pages[r]
        x = (spread * rng.standard_normal((self.slots, hkv, d))).astype(np.float32)
        free = np.setdiff1d(np.arange(self.slots), self.table)
        if kind == "fp4":
            rows = fp4.pack(*fp4.quantise(x, KS))
            rows[free] = 0xFF
            self.pool = torch.from_numpy(rows)
        elif kind == "fp8":
            y = torch.from_numpy(x / np.float32(KS)).to(torch.float8_e4m3fn).view(torch.uint8)
            y[free] = 0x7F
            self.pool = y
        else:
            x[free] = np.nan
            self.pool = torch.from_numpy(x).to(torch.float32 if kind == "f32" else torch.bfloat16)

    def params(self, **kw):
        return sgl.make_params(KINDS[self.kind], self.B, self.hq, self.hkv, self.d, self.slots, k_scale=KS, v_scale=VS, **kw)

    def queries(self, n):
        q = self.rng.standard_normal((n, self.hq, self.d)).astype(np.float32)
        return torch.from_numpy(q).to(torch.float32 if self.kind == "f32" else torch.bfloat16)

    def keys(self, r, n):
        rows = self.pool[self.table[r, :n].astype(np.int64)]
        if self.kind == "fp4":
            c, s = fp4.unpack(rows.numpy(), self.hkv, self.d)
            return KS * fp4.e2m1_to_float(c) * np.repeat(e4m3_to_float(s), 16, -1)
        if self.kind == "fp8":
            return KS * e4m3_to_float(rows.numpy())
        return rows.double().numpy()

    def lse(self, q, pre, ext, sm):
        """Log-sum-exps [N, hq] of rows in request order, row i of request r at position pre[r] + i."""
        out, at = np.full((q.shape[0], self.hq), -np.inf, dtype=np.float32), 0
        x = q.double().numpy()
        for r in range(self.B):
            k = self.keys(r, int(pre[r] + ext[r]))
            for h in range(self.hq):
                if not ext[r]:
                    break
                s = sm * x[at:at + ext[r], h] @ k[:, h * self.hkv // self.hq].T
                s[np.arange(s.shape[1])[None] > pre[r] + np.arange(ext[r])[:, None]] = -np.inf
                m = s.max(1)
                out[at:at + ext[r], h] = m + np.log(np.exp(s - m[:, None]).sum(1))
            at += ext[r]
        return torch.from_numpy(out)

    def expect(self, q, lse, pre, ext, window, scores, decay, decode, sm):
        """(scores, bound): the positions past a context as they were (bound 0)."""
        want, tol = np.full(scores.shape, 7.0), np.zeros(scores.shape)
        x, l, at = q.double().numpy(), lse.double().numpy(), 0
        for r in range(self.B):
            n, L = int(ext[r]), int(pre[r] + ext[r])
            ask = min(n, window) if window else n
            old = np.zeros(L)
            fresh = int(pre[r])
            old[:fresh] = scores[r, :fresh].astype(np.float64) * np.float64(np.float32(decay))
            if L:
                w, b = oevict.weights(x[at + n - ask:at + n], l[at + n - ask:at + n], self.keys(r, L), L - ask, sm)
                want[r, :L] = old + w
                tol[r, :L] = b + 2.0 ** -23 * np.abs(want[r, :L])
            at += n
        return want, tol


def _run(c, q, lse, pre, ext, window, scores, decay, decode, in_place=False, stream=None, ws=None, **kw):
    """The call's scores; scores None: from zeros."""
    p = c.params(**({} if decode else dict(host_prefix_lens=pre, host_extend_lens=ext)), **kw)
    n = sgl.sgl_attn_weights_workspace_bytes(p, window)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda") if ws is None else ws
    lens = torch.from_numpy((pre + ext if decode else pre).astype(np.int32)).cuda()
    extd = None if decode else torch.from_numpy(np.asarray(ext, dtype=np.int32)).cuda()
    si = None if scores is None else torch.from_numpy(scores).cuda()
    shape = (c.B, c.ld) if scores is None else scores.shape
    so = si if in_place else torch.full(shape, 7.0, device="cuda")
    args = (q.cuda(), lse.cuda(), c.pool.cuda(), torch.from_numpy(c.table).cuda(), lens, extd, p, si, so, ws)
    torch.cuda.synchronize()
    sgl.sgl_attn_weights(*args, decay=decay, window=window, stream=stream)
    torch.cuda.synchronize()
    sgl.sgl_check(ws)
    return so.cpu().numpy()


def _check(c, pre, ext, window=0, decay=1.0, decode=False, sld=None, none=False, in_place=False, **kw):
    pre, ext = np.asarray(pre, dtype=np.int64), np.asarray(ext, dtype=np.int64)
    n = c.B if decode else int(ext.sum())
    q = c.queries(n)
    sm = 1 / np.sqrt(c.d)
    if decode:        # (a request without context still has a row)
        lse, full = torch.full((n, c.hq), -np.inf), np.nonzero(ext)[0]
        lse[full] = c.lse(q[full], pre, ext, sm)
    else:
        lse = c.lse(q, pre, ext, sm)
    scores = (4 * c.rng.random((c.B, sld or c.ld))).astype(np.float32)
    got = _run(c, q, lse, pre, ext, window, None if none else scores, decay, decode, in_place, **kw)
    if none and sld is None:
        scores = np.zeros_like(scores)
    rows = q[full] if decode else q
    want, tol = c.expect(rows, lse[full] if decode else lse, pre, ext, window, scores, 0.0 if none else decay, decode, sm)
    if in_place:
        L = pre + ext
        past = np.arange(want.shape[1])[None] >= L[:, None]
        want = np.where(past, scores, want)
    err = np.abs(got.astype(np.float64) - want)
    assert (err <= tol).all(), "worst %.3g of the bound, at %s" % ((err / np.maximum(tol, 1e-30)).max(),
                                                                   np.argwhere(err > tol)[:4].tolist())
    return got


# ------------------------------------------------------------------ decode
@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_decode(kind, hq, hkv, d):
    lens = np.array([1, 2, 15, 16, 17, 0, 31, 32, 33, 63, 64, 65, 127, 129, 300, 1000])
    c = Cache(kind, lens, hq, hkv, d, ld=1003, seed=hq + d)
    has = (lens > 0).astype(np.int64)
    _check(c, lens - has, has, decode=True)
    _check(c, lens - has, has, decode=True, decay=0.5, sld=1001)
    _check(c, lens - has, has, decode=True, decay=0.0)
    _check(c, lens - has, has, decode=True, none=True)
    _check(c, lens - has, has, decode=True, decay=0.75, in_place=True)


@pytest.mark.parametrize("kind", list(KINDS))
def test_decode_of_many_requests_and_of_long_ones(kind):
    rng = np.random.default_rng(1)
    lens = rng.integers(0, 90, 333)
    has = (lens > 0).astype(np.int64)
    _check(Cache(kind, lens, 4, 2, 64, seed=1), lens - has, has, decode=True)
    lens = np.array([20011, 3, 7000])
    _check(Cache(kind, lens, 8, 2, 128, page=16, seed=2), lens - 1, np.ones(3, dtype=np.int64), decode=True, decay=0.9)


# ------------------------------------------------------------------ chunks
@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_chunks(kind, hq, hkv, d):
    pre, ext = np.array([0, 0, 5, 100, 0, 130, 257, 64, 40]), np.array([1, 33, 1, 70, 0, 2, 150, 64, 0])
    c = Cache(kind, pre + ext, hq, hkv, d, ld=410, seed=hq + d)
    for window in (0, 1, 8, 33, 1000):
        _check(c, pre, ext, window)
    _check(c, pre, ext, decay=0.5, sld=409)
    _check(c, pre, ext, 5, none=True)
    _check(c, pre, ext, 0, decay=0.25, in_place=True)


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (8, 1, 64), (5, 5, 128)])
def test_long_chunks(kind, hq, hkv, d):
    pre, ext = np.array([700, 0, 129]), np.array([260, 515, 128])
    c = Cache(kind, pre + ext, hq, hkv, d, page=16, seed=3)
    _check(c, pre, ext)
    _check(c, pre, ext, 100, decay=0.0)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,n", [(2, 2, 11000), (8, 1, 9100)])
def test_long_prompts_from_the_start(kind, hq, hkv, n):
    """More than 32 tiles that only some runs of query blocks see.  Against float64 on the GPU; a score sums n hq weights
    in fp32, off by 2^-24 of itself for each of them at most, the weights themselves by less than 2^-13 (a product's sum of
    magnitudes is below 2^5 here: 2^5 (64 + 12) 2^-24, and 2^-21)."""
    c = Cache(kind, [n, 300], hq, hkv, 64, seed=n)
    pre, ext = np.array([0, 100]), np.array([n, 200])
    q = c.queries(n + 200)
    want, lse, at = np.zeros((2, n)), torch.zeros(n + 200, hq, dtype=torch.float64, device="cuda"), 0
    for r in range(2):
        L, e = int(pre[r] + ext[r]), int(ext[r])
        k, x = torch.from_numpy(c.keys(r, L)).cuda(), q[at:at + e].double().cuda()
        hidden = torch.arange(L, device="cuda")[None] > int(pre[r]) + torch.arange(e, device="cuda")[:, None]
        for h in range(hq):
            w = (x[:, h] @ k[:, h * hkv // hq].T / 8).masked_fill_(hidden, -torch.inf)
            lse[at:at + e, h] = torch.logsumexp(w, 1).float().double()
            want[r, :L] += w.sub_(lse[at:at + e, h, None]).exp_().sum(0).cpu().numpy()
        at += e
    got = _run(c, q, lse.float().cpu(), pre, ext, 0, None, 1.0, False)
    for r in range(2):
        L = int(pre[r] + ext[r])
        err = np.abs(got[r, :L] - want[r, :L])
        assert (err <= want[r, :L] * ((int(ext[r]) * hq + 8) * 2.0 ** -24 + 2.0 ** -13) + 1e-30).all(), err.max()


@pytest.mark.parametrize("kind", list(KINDS))
def test_chunks_of_many_requests(kind):
    rng = np.random.default_rng(4)
    ext, pre = rng.integers(0, 9, 300), rng.integers(0, 60, 300)
    c = Cache(kind, pre + ext, 8, 2, 64, seed=4)
    _check(c, pre, ext)
    _check(c, pre, ext, 2)


@pytest.mark.parametrize("kind", list(KINDS))
def test_weights_of_every_row_sum_to_one(kind):
    """The weights that a request's tokens get from the attention calls' own log-sum-exps, chunk and decode: one for
    each asking row and head, to the bounds of both."""
    hq, hkv, d = 16, 4, 128
    pre, ext = np.array([0, 200, 77]), np.array([150, 40, 1])
    c = Cache(kind, pre + ext, hq, hkv, d, seed=8)
    q = c.queries(int(ext.sum()))
    p = c.params(host_prefix_lens=pre, host_extend_lens=ext)
    ws = torch.zeros(max(256, sgl.sgl_extend_workspace_bytes(p)), dtype=torch.uint8, device="cuda")
    v = torch.zeros_like(c.pool).cuda()
    lse, o = torch.zeros(len(q), hq, device="cuda"), torch.zeros_like(q).cuda()
    pd, ed = (torch.from_numpy(x.astype(np.int32)).cuda() for x in (pre, ext))
    table = torch.from_numpy(c.table).cuda()
    sgl.sgl_extend_attn(q.cuda(), c.pool.cuda(), v, table, pd, ed, p, o, lse, ws)
    sgl.sgl_check(ws)
    got = _run(c, q, lse.cpu(), pre, ext, 0, None, 1.0, False)
    for r in range(3):
        L = int(pre[r] + ext[r])
        # log-sum-exps are good to 2e-5 here (fp32 sums of a few hundred weights of scores below 2^5)
        assert abs(got[r, :L].astype(np.float64).sum() / (ext[r] * hq) - 1) < 3e-5


# ------------------------------------------------------------------ what is masked, missing or odd
@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("window", [0, 4])
def test_a_nan_key_reaches_its_own_token_only(kind, window):
    pre, ext = np.array([100, 0]), np.array([60, 140])
    c = Cache(kind, pre + ext, 8, 2, 64, seed=6)
    q = c.queries(int(ext.sum()))
    lse = c.lse(q, pre, ext, 0.125)
    clean = _run(c, q, lse, pre, ext, window, None, 1.0, False)
    at = [(0, 3), (0, 99), (0, 100), (0, 158), (1, 0), (1, 139)]
    for r, p in at:
        slot = int(c.table[r, p])
        if kind == "fp4":
            codes, sf = fp4.unpack(c.pool.numpy(), 2, 64)
            sf[slot, 1, 2] = 0x7F
            c.pool = torch.from_numpy(fp4.pack(codes, sf))
        elif kind == "fp8":
            c.pool[slot, 1, 33] = 0x7F
        else:
            c.pool[slot, 1, 33] = float("nan")
    got = _run(c, q, lse, pre, ext, window, None, 1.0, False)
    hit = np.zeros(got.shape, dtype=bool)
    hit[tuple(np.array(at).T)] = True
    assert np.isnan(got[hit]).all() and np.array_equal(got[~hit], clean[~hit])


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("decode", [False, True])
def test_rows_without_a_sum_and_rows_of_nan(kind, decode):
    ext = np.array([1, 1, 1]) if decode else np.array([40, 3, 70])
    pre = np.array([150, 20, 9])
    c = Cache(kind, pre + ext, 8, 4, 64, seed=7)
    q = c.queries(int(ext.sum()))
    lse = c.lse(q, pre, ext, 0.125)
    a = lse.clone()
    first = np.cumsum(ext) - ext
    a[first[0]] = -np.inf                         # this row adds nothing
    a[first[1], 2] = -np.inf
    got = _run(c, q, a, pre, ext, 0, None, 1.0, decode)
    want, tol = c.expect(q, a, pre, ext, 0, np.zeros(got.shape, dtype=np.float32), 0.0, decode, 0.125)
    assert (np.abs(got - want) <= tol).all()
    b = lse.clone()
    b[first[2], 1] = np.nan                       # every token that it sees, and no other
    got = _run(c, q, b, pre, ext, 0, None, 1.0, decode)
    clean = _run(c, q, lse, pre, ext, 0, None, 1.0, decode)
    sees = int(pre[2]) + 1
    assert np.isnan(got[2, :sees]).all()
    got[2, :sees] = clean[2, :sees]
    assert np.array_equal(got, clean)


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("decode", [False, True])
def test_bad_slots_and_lengths_are_reported(kind, decode):
    ext = np.array([1, 1, 1]) if decode else np.array([40, 3, 70])
    pre = np.array([150, 20, 9])
    c = Cache(kind, pre + ext, 8, 4, 64, ld=200, seed=7)
    q = c.queries(int(ext.sum()))
    lse = c.lse(q, pre, ext, 0.125)
    scores = (4 * c.rng.random((3, 200))).astype(np.float32)
    clean = _run(c, q, lse, pre, ext, 0, scores, 0.5, decode)
    good = c.table.copy()
    for (r, p), bad in (((0, 7), c.slots), ((1, 20), -1), ((2, 9), 2 ** 31 - 1), ((0, 150), -2 ** 31)):
        c.table[r, p] = bad
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    with pytest.raises(sgl.SglError) as e:
        _run(c, q, lse, pre, ext, 0, scores, 0.5, decode, ws=ws)
    assert e.value.status == -5
    # the same call's scores: these tokens get no weight, the others what they got
    lens = torch.from_numpy((pre + ext if decode else pre).astype(np.int32)).cuda()
    extd = None if decode else torch.from_numpy(ext.astype(np.int32)).cuda()
    p = c.params(**({} if decode else dict(host_prefix_lens=pre, host_extend_lens=ext)))

    def run(lens, table):
        out = torch.full((3, 200), 7.0, device="cuda")
        sgl.sgl_attn_weights(q.cuda(), lse.cuda(), c.pool.cuda(), torch.from_numpy(table).cuda(), lens, extd, p,
                             torch.from_numpy(scores).cuda(), out, ws, decay=0.5)
        with pytest.raises(sgl.SglError):
            sgl.sgl_check(ws)
        return out.cpu().numpy()
    got = run(lens, c.table)
    for (r, x) in ((0, 7), (1, 20), (2, 9), (0, 150)):
        old = np.float32(0.5) * scores[r, x] if x < pre[r] else np.float32(0)
        assert got[r, x] == old, (r, x)
        got[r, x] = clean[r, x]
    assert np.array_equal(got, clean)
    # a length that the tables do not hold: that request's scores stay as they were
    for bad in (201, -1, 2 ** 31 - 1):
        l2 = lens.clone()
        l2[1] = bad
        got = run(l2, good)
        assert (got[1] == 7).all() and np.array_equal(got[[0, 2]], clean[[0, 2]])


@pytest.mark.parametrize("kind", ["fp8", "fp4"])
def test_a_query_beyond_f16(kind):
    """A decode batch over FP8 or 4-bit keys reports it; chunks multiply in bf16 and take it as it is."""
    pre, ext = np.array([150, 20]), np.array([1, 1])
    c = Cache(kind, pre + ext, 8, 4, 64, seed=7)
    q = c.queries(2)
    q[-1, 3, 17] = 70000.0
    lse = c.lse(q, pre, ext, 0.125)
    with pytest.raises(sgl.SglError) as e:
        _run(c, q, lse, pre, ext, 0, None, 1.0, True)
    assert e.value.status == -5
    got = _run(c, q, lse, pre, ext, 0, None, 1.0, False)
    want, tol = c.expect(q, lse, pre, ext, 0, np.zeros(got.shape, dtype=np.float32), 0.0, False, 0.125)
    assert (np.abs(got - want) <= tol).all()


@pytest.mark.parametrize("kind", list(KINDS))
def test_the_same_bits_again_and_on_another_stream(kind):
    pre, ext = np.array([300, 0, 77, 900]), np.array([80, 260, 1, 33])
    c = Cache(kind, pre + ext, 32, 8, 128, seed=9)
    q = c.queries(int(ext.sum()))
    lse = c.lse(q, pre, ext, 1 / np.sqrt(128))
    a = _run(c, q, lse, pre, ext, 0, None, 1.0, False)
    for s in (None, torch.cuda.Stream()):
        assert np.array_equal(_run(c, q, lse, pre, ext, 0, None, 1.0, False, stream=s), a)
    one = np.ones(4, dtype=np.int64)
    a = _run(c, q[:4], lse[:4], pre + ext - 1, one, 0, None, 1.0, True)
    for s in (None, torch.cuda.Stream()):
        assert np.array_equal(_run(c, q[:4], lse[:4], pre + ext - 1, one, 0, None, 1.0, True, stream=s), a)


@pytest.mark.parametrize("kind", ["bf16", "fp4"])
def test_decode_in_a_graph_follows_the_lengths(kind):
    lens = np.array([5, 130, 0, 64])
    c = Cache(kind, lens + 6, 8, 2, 128, ld=140, seed=10)
    q, sm = c.queries(4), 1 / np.sqrt(128)
    qd, pool, table = q.cuda(), c.pool.cuda(), torch.from_numpy(c.table).cuda()
    lse = torch.zeros(4, 8, device="cuda")
    scores = torch.zeros(4, 140, device="cuda")
    dl = torch.from_numpy(lens.astype(np.int32)).cuda()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    p = c.params()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            sgl.sgl_attn_weights(qd, lse, pool, table, dl, None, p, scores, scores, ws)
    total = np.zeros((4, 140))
    tol = np.zeros((4, 140))
    for step in range(4):
        n = lens + step
        x = c.lse(q[n > 0], n - (n > 0), (n > 0).astype(np.int64), sm)
        lse[torch.from_numpy(n > 0).cuda()] = x.cuda()
        dl.copy_(torch.from_numpy(n.astype(np.int32)))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want, b = c.expect(q[n > 0], x, n - (n > 0), (n > 0).astype(np.int64), 0, total.astype(np.float32), 1.0, True, sm)
        live = np.arange(140)[None] < n[:, None]
        assert (np.abs(scores.cpu().numpy() - want) <= b)[live].all()
        total = scores.cpu().numpy().astype(np.float64)
    sgl.sgl_check(ws)
    assert not scores.cpu().numpy()[np.arange(140)[None] >= (lens + 3)[:, None]].any() and tol.sum() == 0


@pytest.mark.parametrize("kind,hkv", [("bf16", 8), ("f32", 8), ("fp8", 16), ("fp4", 32)])
@pytest.mark.parametrize("decode", [False, True])
def test_rows_far_into_the_pool(kind, hkv, decode):
    """Keys more than 2^31 bytes into a pool."""
    pre, ext = np.array([30, 0]), np.array([1, 1]) if decode else np.array([40, 5])
    c = Cache(kind, pre + ext, hkv, hkv, 128, seed=13)
    q = c.queries(int(ext.sum()))
    lse = c.lse(q, pre, ext, 128 ** -0.5)
    near = _run(c, q, lse, pre, ext, 0, None, 1.0, decode)
    first = 2 ** 31 // (c.pool[0].numel() * c.pool.element_size()) + 5
    far = torch.zeros(first + c.slots, *c.pool.shape[1:], dtype=c.pool.dtype, device="cuda")
    far[first:] = c.pool.cuda()
    table = torch.from_numpy(np.where(c.table >= 0, c.table + first, -1).astype(np.int32)).cuda()
    c.slots += first
    p = c.params(**({} if decode else dict(host_prefix_lens=pre, host_extend_lens=ext)))
    ws = torch.zeros(sgl.sgl_attn_weights_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    lens = torch.from_numpy((pre + ext if decode else pre).astype(np.int32)).cuda()
    extd = None if decode else torch.from_numpy(ext.astype(np.int32)).cuda()
    out = torch.full(near.shape, 7.0, device="cuda")
    sgl.sgl_attn_weights(q.cuda(), lse.cuda(), far, table, lens, extd, p, None, out, ws)
    sgl.sgl_check(ws)
    assert np.array_equal(out.cpu().numpy(), near)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_two_streams_at_once(kind):
    """Two chunk calls side by side, each with its workspace: the bits of each alone."""
    runs = []
    for seed, (pre, ext) in enumerate((([900, 40], [200, 130]), ([10, 700], [300, 64]))):
        pre, ext = np.array(pre), np.array(ext)
        c = Cache(kind, pre + ext, 16, 4, 128, seed=seed)
        q = c.queries(int(ext.sum()))
        lse = c.lse(q, pre, ext, 128 ** -0.5)
        alone = _run(c, q, lse, pre, ext, 0, None, 1.0, False)
        p = c.params(host_prefix_lens=pre, host_extend_lens=ext)
        ws = torch.zeros(sgl.sgl_attn_weights_workspace_bytes(p), dtype=torch.uint8, device="cuda")
        out = torch.full(alone.shape, 7.0, device="cuda")
        pd, ed = (torch.from_numpy(x.astype(np.int32)).cuda() for x in (pre, ext))
        runs.append((torch.cuda.Stream(), alone, out, ws,
                     (q.cuda(), lse.cuda(), c.pool.cuda(), torch.from_numpy(c.table).cuda(), pd, ed, p, None, out, ws)))
    torch.cuda.synchronize()
    for _ in range(20):
        for s, _, _, _, args in runs:
            sgl.sgl_attn_weights(*args, stream=s)
    torch.cuda.synchronize()
    for _, alone, out, ws, _ in runs:
        sgl.sgl_check(ws)
        assert np.array_equal(out.cpu().numpy(), alone)


@pytest.mark.parametrize("kind", ["bf16", "fp4"])
def test_a_captured_chunk_with_the_eviction_behind_it(kind):
    """Weights of a chunk and the eviction by them in one graph, replayed without waits in between."""
    pre, ext = np.array([300, 0, 150]), np.array([60, 200, 33])
    c = Cache(kind, pre + ext, 8, 2, 128, ld=400, seed=14)
    q = c.queries(int(ext.sum()))
    lse = c.lse(q, pre, ext, 128 ** -0.5)
    p = c.params(host_prefix_lens=pre, host_extend_lens=ext)
    ws = torch.zeros(sgl.sgl_attn_weights_workspace_bytes(p, 16), dtype=torch.uint8, device="cuda")
    pd, ed, n = (torch.from_numpy(x.astype(np.int32)).cuda() for x in (pre, ext, pre + ext))
    table = torch.from_numpy(c.table).cuda()
    scores, kept, to, lens = torch.zeros(3, 400, device="cuda"), torch.zeros(3, 400, device="cuda"), table.clone(), n.clone()
    bud = torch.full((3,), 100, dtype=torch.int32, device="cuda")
    qd, ld, pool = q.cuda(), lse.cuda(), c.pool.cuda()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            sgl.sgl_attn_weights(qd, ld, pool, table, pd, ed, p, None, scores, ws, window=16)
            sgl.sgl_kv_evict(scores, table, n, bud, kept, to, lens, ws, recent=16)
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    sgl.sgl_check(ws)
    sc = scores.cpu().numpy()
    want, tol = c.expect(q, lse, pre, ext, 16, np.zeros((3, 400), dtype=np.float32), 0.0, False, 128 ** -0.5)
    for r in range(3):
        L = int(pre[r] + ext[r])
        assert (np.abs(sc[r, :L] - want[r, :L]) <= tol[r, :L]).all()
        stays = oevict.keep(sc[r, :L], 100, recent=16)
        assert int(lens[r]) == 100 and np.array_equal(to[r, :100].cpu().numpy(), c.table[r, :L][stays])
        assert np.array_equal(kept[r, :100].cpu().numpy(), sc[r, :L][stays])


def test_python_arguments_are_checked():
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    lse, sc = torch.zeros(4, 2, device="cuda"), torch.zeros(4, 8, device="cuda")
    pool = torch.zeros(16, 2, 64, dtype=torch.bfloat16, device="cuda")
    t = torch.zeros(4, 8, dtype=torch.int32, device="cuda")
    n = torch.zeros(4, dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    p = sgl.make_params(sgl.SGL_DTYPE_BF16, 4, 2, 2, 64, 16)
    good = dict(q=q, lse=lse, k_pool=pool, req_to_token=t, lens=n, extend_lens=None, params=p, scores_in=sc, scores_out=sc,
                workspace=ws)
    for bad in (dict(q=q.float()), dict(q=q[:3]), dict(q=q.transpose(0, 1)), dict(lse=lse[:3]), dict(lse=lse.double()),
                dict(k_pool=pool[:15]), dict(req_to_token=t.long()), dict(req_to_token=t[:3]), dict(lens=n[:3]),
                dict(extend_lens=n), dict(scores_in=sc[:, :4].contiguous()), dict(scores_out=sc.double()),
                dict(scores_out=sc.cpu()), dict(workspace=ws.cpu())):
        with pytest.raises((TypeError, ValueError)):
            sgl.sgl_attn_weights(**dict(good, **bad))
    for bad in (dict(decay=-1.0), dict(decay=float("nan")), dict(decay=float("inf")), dict(window=-1),
                dict(workspace=ws[:128])):
        with pytest.raises(sgl.SglError):
            sgl.sgl_attn_weights(**dict(good, **bad))
    few = sgl.make_params(sgl.SGL_DTYPE_BF16, 4, 2, 2, 64, 16, host_prefix_lens=[0] * 4, host_extend_lens=[2] * 4)
    with pytest.raises(ValueError):               # rows of eight new tokens in a tensor of four
        sgl.sgl_attn_weights(**dict(good, extend_lens=n, params=few))
    sgl.sgl_attn_weights(**good)
    sgl.sgl_check(ws)
    assert not sc.any()


# ------------------------------------------------------------------ the loop
@pytest.mark.parametrize("kind", list(KINDS))
def test_a_cache_thinned_out_while_it_decodes(kind):
    """Prompts are appended and attended to, scored by their last rows and cut to a budget; then each step appends a
    token at its true position, attends, adds weights and gives a token back.  The device's own selections are
    followed: each is checked against the oracle's on the device's scores, each result against float64 over the pool's
    contents and the kept tokens."""
    hq, hkv, d, B, budget, recent = 8, 2, 64, 3, 40, 6
    prompt = np.array([100, 64, 41])
    ld, slots = 128, 512
    c = Cache(kind, [0] * B, hq, hkv, d, ld=ld, seed=11)
    c.slots = slots
    g = torch.Generator().manual_seed(12)
    dt = torch.float32 if kind == "f32" else torch.bfloat16
    if kind == "fp4":
        kp, vp = (torch.full((slots, fp4.row_bytes(hkv, d)), 0xFF, dtype=torch.uint8, device="cuda") for _ in "kv")
    elif kind == "fp8":
        kp, vp = (torch.full((slots, hkv, d), 0x7F, dtype=torch.uint8, device="cuda") for _ in "kv")
    else:
        kp, vp = (torch.full((slots, hkv, d), float("nan"), dtype=dt, device="cuda") for _ in "kv")
    rope = sgl.sgl_rope_create(d, axes=(12, 10, 10))
    tree = sgl.sgl_tree_create(slots, 1, np.random.default_rng(3).permutation(slots).astype(np.int32))
    own = [set() for _ in range(B)]
    table = np.full((B, ld), -1, dtype=np.int32)
    for r in range(B):
        s = sgl.sgl_tree_alloc(tree, int(prompt[r]))
        table[r, :prompt[r]] = s
        own[r] |= set(s.tolist())
    td = torch.from_numpy(table).cuda()
    lens = torch.from_numpy(prompt.astype(np.int32)).cuda()
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    scores, posr = torch.zeros(B, ld, device="cuda"), torch.zeros(B, ld, dtype=torch.int32, device="cuda")
    for r in range(B):
        posr[r, :prompt[r]] = torch.arange(int(prompt[r]), dtype=torch.int32)
    bud = torch.full((B,), budget, dtype=torch.int32, device="cuda")
    ev, cnt = torch.zeros(B, ld, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")

    def new(n):
        return [torch.randn(n, h, d, generator=g).to(dt).cuda() for h in (hq, hkv, hkv)]

    def evict():
        before = [x.cpu().numpy().copy() for x in (scores, td, posr, lens)]
        sgl.sgl_kv_evict(scores, td, lens, bud, scores, td, lens, ws, ev, cnt, posr, posr, sinks=2, recent=recent)
        sgl.sgl_check(ws)
        for r in range(B):
            n = int(before[3][r])
            stays = oevict.keep(before[0][r, :n], budget, 1, 2, recent)
            assert int(lens[r]) == int(stays.sum())
            for x, y in ((scores, before[0]), (td, before[1]), (posr, before[2])):
                assert np.array_equal(x[r, :int(stays.sum())].cpu().numpy(), y[r, :n][stays])
            gone = ev[r, :int(cnt[r])].cpu().numpy()
            assert np.array_equal(gone, before[1][r, :n][~stays])
            own[r] -= set(gone.tolist())
            if len(gone):
                sgl.sgl_tree_free(tree, gone)

    def hold(pre, ext, q, o, lse, before, window, decode):
        """Outputs and scores against float64 over what the pool holds."""
        c.table, c.pool = td.cpu().numpy(), kp.cpu()
        want, tol = c.expect(q.cpu(), lse.cpu(), pre, ext, window, before, 1.0, decode, 0.125)
        got = scores.cpu().numpy()
        live = np.arange(ld)[None] < (pre + ext)[:, None]
        assert (np.abs(got - want) <= tol)[live].all()
        ref = c.lse(q.cpu(), pre, ext, 0.125).numpy()
        assert np.abs(lse.cpu().numpy() - ref).max() < 1e-3

    # the prompts: text positions on axis 0, a picture's rows and columns on the others
    n = int(prompt.sum())
    q, k, v = new(n)
    places = torch.stack([torch.cat([torch.arange(int(x)) for x in prompt]), torch.arange(n) % 7, torch.arange(n) % 5])
    p = c.params(host_prefix_lens=[0] * B, host_extend_lens=prompt)
    ws = torch.zeros(max(256, sgl.sgl_attn_weights_workspace_bytes(p, 8)), dtype=torch.uint8, device="cuda")
    qo = torch.empty_like(q)
    sgl.sgl_kv_append_at(rope, p, q, k, v, kp, vp, td, zero, lens, places.to(torch.int32).cuda(), qo, ws)
    o, lse = torch.empty_like(q), torch.empty(n, hq, device="cuda")
    sgl.sgl_extend_attn(qo, kp, vp, td, zero, lens, p, o, lse, ws)
    sgl.sgl_attn_weights(qo, lse, kp, td, zero, lens, p, None, scores, ws, window=8)
    sgl.sgl_check(ws)
    hold(np.zeros(B, dtype=np.int64), prompt, qo, o, lse, np.zeros((B, ld), dtype=np.float32), 8, False)
    evict()
    assert lens.tolist() == [budget] * B
    # steps: the rows no longer count the tokens, positions are given
    for step in range(3):
        host = lens.cpu().numpy().astype(np.int64)
        row = td.cpu().numpy()
        for r in range(B):
            s = sgl.sgl_tree_alloc(tree, 1)
            row[r, host[r]] = s[0]
            own[r].add(int(s[0]))
            posr[r, int(host[r])] = int(prompt[r]) + step
        td.copy_(torch.from_numpy(row))
        lens += 1
        q, k, v = new(B)
        at = torch.from_numpy(prompt + step).to(torch.int32).repeat(3, 1).cuda()
        qo, lse, o = torch.empty_like(q), torch.empty(B, hq, device="cuda"), torch.empty_like(q)
        grp = sgl.sgl_groups_create()
        sgl.sgl_groups_from_table(row, (host + 1).astype(np.int32), grp)
        pd = c.params()
        plan = sgl.sgl_decode_plan(pd, (host + 1).astype(np.int32), sgl.sgl_groups_view(grp))
        sgl.sgl_groups_destroy(grp)
        wd = torch.zeros(max(256, plan.workspace_bytes), dtype=torch.uint8, device="cuda")
        sgl.sgl_plan_upload(plan, wd)
        before = scores.cpu().numpy().copy()
        sgl.sgl_kv_append_at(rope, pd, q, k, v, kp, vp, td, lens, None, at, qo, wd)
        sgl.sgl_decode_attn(qo, kp, vp, td, lens, plan, o, lse, wd)
        sgl.sgl_attn_weights(qo, lse, kp, td, lens, None, pd, scores, scores, wd)
        sgl.sgl_check(wd)
        # the rotated query, at its true position on every axis
        freq = orope.frequencies(d, 10000.0)
        ref = orope.rotate(q.double().cpu().numpy(), (prompt + step).astype(np.float64), freq)
        assert np.abs(qo.double().cpu().numpy() - ref).max() < 0.05
        hold(host, np.ones(B, dtype=np.int64), qo, o, lse, before, 0, True)
        evict()
        assert lens.tolist() == [budget] * B
    for r in range(B):
        assert set(td[r, :budget].tolist()) == own[r]
    assert sgl.sgl_tree_stats(tree)["free_pages"] == slots - B * budget
    sgl.sgl_tree_destroy(tree)
