"""Attention over a 4-bit cache on the GPU against float64 attention over the
pool's dequantised values, and the run append -> decode / extend.

Bounds, per output element (A = the attention-weighted mean of |V|, L = the
context's length): scores are fp32 sums of exact products, off by at most
delta = sm_scale * max_j sum_i |q_i K_ji| * (d + 8) 2^-24 + 2^-21 (the last term:
the scaling and the exponential), which changes weights by a factor within
2 delta; weights enter the second product as f16, off by 2^-11 of themselves,
or by 2^-25 below f16's normal range (against a sum of at least one); the
output is rounded to bf16, half a step being 2^-8 of the value.  So
  |O - O64| <= 2^-8 |O64| + (1 + 2^-8) ((2^-11 + 2 delta) A + L 2^-25 max |V|)
  |LSE - LSE64| <= delta + (L + 64) 2^-24 + 2^-23 |LSE64|.
"""

import numpy as np
import pytest
import torch

import radixattention_prefix_shared_radix_gb300 as sgl
from oracle import fp4, rope as orope

pytestmark = pytest.mark.gpu

KS, VS = 0.37, 1.3


@pytest.fixture(scope="module", autouse=True)
def _built():
    from radixattention_prefix_shared_radix_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def _pool(slots, hkv, d, scale, seed, used=None):
    """A 4-bit pool of quantised normal values; slots outside `used` hold NaN scales and arbitrary codes."""
    rng = np.random.default_rng(seed)
    rows = fp4.pack(*fp4.quantise(rng.standard_normal((slots, hkv, d)).astype(np.float32), scale))
    if used is not None:
        rest = np.ones(slots, dtype=bool)
        rest[used] = False
        rows[rest] = 0xFF
    return rows


def _ref(q, kv, vv, sm, k_pre=None):
    """One query row [Hq, d] over K, V [L, Hkv, d]: (O, LSE, their bounds)."""
    hq, d = q.shape
    L, hkv = kv.shape[:2]
    G = hq // hkv
    O, lse = np.zeros((hq, d)), np.full(hq, -np.inf)
    to, tl = np.zeros((hq, d)), np.zeros(hq)
    if L == 0:
        return O, lse, to, tl
    for h in range(hkv):
        qq = q[h * G:(h + 1) * G]
        s = sm * qq @ kv[:, h].T
        size = sm * (np.abs(qq) @ np.abs(kv[:, h]).T).max(1)
        m = s.max(1, keepdims=True)
        w = np.exp(s - m)
        l = w.sum(1, keepdims=True)
        w /= l
        sl = slice(h * G, (h + 1) * G)
        O[sl], lse[sl] = w @ vv[:, h], (m + np.log(l))[:, 0]
        delta = (size * (d + 8) * 2.0 ** -24 + 2.0 ** -21)[:, None]
        to[sl] = 2.0 ** -8 * np.abs(O[sl]) + (1 + 2.0 ** -8) * (
            (2.0 ** -11 + 2 * delta) * (w @ np.abs(vv[:, h])) + L * 2.0 ** -25 * np.abs(vv[:, h]).max())
        tl[sl] = delta[:, 0] + (L + 64) * 2.0 ** -24 + 2.0 ** -23 * np.abs(lse[sl])
    return O, lse, to, tl


def _close(O, lse, ref):
    Or, lr, to, tl = ref
    assert np.array_equal(np.isneginf(lse), np.isneginf(lr))
    fin = np.isfinite(lr)
    err = np.abs(O - Or)
    assert (err <= to).all(), "O: worst %.3g of the bound" % (err / np.maximum(to, 1e-30)).max()
    el = np.abs(lse[fin] - lr[fin])
    assert (el <= tl[fin]).all(), "LSE: worst %.3g of the bound" % (el / tl[fin]).max()


class Batch:
    """Requests as chains of shared segments over a paged 4-bit pool."""

    def __init__(self, chains, hq, hkv, d, page=1, seed=0, extra=0):
        # chains: per request a list of (segment name, length); equal names share slots
        rng = np.random.default_rng(seed)
        lens = [sum(n for _, n in c) for c in chains]
        B, self.ld = len(chains), max(max(lens, default=1), 1) + extra
        need = {}
        for c in chains:
            for name, n in c:
                need[name] = n
        pages = {k: -(-n // page) for k, n in need.items()}
        total = sum(pages.values()) + B * (extra // page + 2)
        self.slots = (total + total // 4 + 8) * page
        order = rng.permutation(self.slots // page)
        at, where = 0, {}
        for k, p in pages.items():
            where[k] = (order[at:at + p, None] * page + np.arange(page)).reshape(-1)[:need[k]]
            at += p
        self.free = (order[at:, None] * page + np.arange(page)).reshape(-1)
        self.table = np.full((B, self.ld), -1, dtype=np.int32)
        for r, c in enumerate(chains):
            row = np.concatenate([where[k] for k, _ in c]) if c else np.zeros(0, dtype=np.int64)
            self.table[r, :len(row)] = row
        self.lens = np.array(lens, dtype=np.int32)
        self.hq, self.hkv, self.d, self.B = hq, hkv, d, B
        used = np.unique(self.table[self.table >= 0])
        self.kp, self.vp = (_pool(self.slots, hkv, d, s, seed + i, used) for i, s in ((1, KS), (2, VS)))
        self.q = torch.from_numpy(rng.standard_normal((B, hq, d)).astype(np.float32)).bfloat16()
        self.page = page

    def params(self, **kw):
        return sgl.make_params(sgl.SGL_DTYPE_BF16_FP4KV, self.B, self.hq, self.hkv, self.d, self.slots, self.page,
                               k_scale=KS, v_scale=VS, **kw)

    def plan(self, **kw):
        g = sgl.sgl_groups_create()
        sgl.sgl_groups_from_table(self.table, self.lens, g)
        p = sgl.sgl_decode_plan(self.params(**kw), self.lens, sgl.sgl_groups_view(g))
        sgl.sgl_groups_destroy(g)
        return p

    def device(self):
        return [torch.from_numpy(x).cuda() for x in (self.kp, self.vp, self.table, self.lens)]

    def run(self, check=True, table=None, **kw):
        plan = self.plan(**kw)
        ws = torch.zeros(max(plan.workspace_bytes, 256), dtype=torch.uint8, device="cuda")
        sgl.sgl_plan_upload(plan, ws)
        kp, vp, t, lens = self.device()
        if table is not None:
            t = torch.from_numpy(table).cuda()
        o = torch.full((self.B, self.hq, self.d), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((self.B, self.hq), 7.0, device="cuda")
        sgl.sgl_decode_attn(self.q.cuda(), kp, vp, t, lens, plan, o, lse, ws)
        if check:
            sgl.sgl_check(ws)
        self.info = sgl.sgl_plan_info(plan)
        out = o.double().cpu().numpy(), lse.double().cpu().numpy()
        return out if check else out + (ws,)

    def ref(self, r, q=None, skip=(), length=None, kp=None, vp=None, table=None, sm=None):
        n = int(self.lens[r]) if length is None else length
        slots = np.delete((self.table if table is None else table)[r, :n], list(skip))
        k = fp4.values((self.kp if kp is None else kp)[slots], self.hkv, self.d, KS)
        v = fp4.values((self.vp if vp is None else vp)[slots], self.hkv, self.d, VS)
        q = self.q[r] if q is None else q
        return _ref(q.double().numpy(), k, v, 1 / np.sqrt(self.d) if sm is None else sm)

    def check(self, out, rows=None, **kw):
        for r in range(self.B) if rows is None else rows:
            _close(out[0][r], out[1][r], self.ref(r, **kw))


def _star(n, prefix, lo, hi, seed=1):
    rng = np.random.default_rng(seed)
    return [[("p", prefix), (r, int(rng.integers(lo, hi + 1)))] for r in range(n)]


def _own(lens):
    return [[(r, n)] if n else [] for r, n in enumerate(lens)]


def _families(sizes, shared, own):
    return [[("f%d" % f, shared), ((f, i), own)] for f, n in enumerate(sizes) for i in range(n)]


EDGE = [[("a", 250)], [], [("b", 1)], [("a", 250), ("c", 3)], [("a", 250)], [("d", 32)], [("e", 31)], [("f", 33)], [],
        [("g", 64), ("h", 1)], [("g", 64)]]


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (8, 8, 64), (16, 2, 64), (8, 1, 64), (8, 1, 128), (40, 5, 128),
                                      (12, 12, 64), (36, 9, 128), (16, 4, 128), (22, 11, 64)])
@pytest.mark.parametrize("shape", ["star", "own", "families", "edge"])
def test_decode(hq, hkv, d, shape):
    chains = {"star": _star(9, 300, 5, 130), "own": _own([700, 0, 1, 31, 32, 33, 65, 128, 511]),
              "families": _families([2, 4, 1, 3, 7], 150, 40), "edge": EDGE}[shape]
    b = Batch(chains, hq, hkv, d, page=16 if shape == "own" else 1, seed=hq + d)
    b.check(b.run())


@pytest.mark.parametrize("num_sms", [1, 5, 152, 1000])
@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (16, 2, 64)])
def test_decode_for_other_targets(num_sms, hq, hkv, d):
    """Other cuts into pieces, down to every piece on one CTA's streams."""
    b = Batch(_star(20, 500, 1, 300) + _families([4, 2], 90, 33) + EDGE, hq, hkv, d, seed=num_sms)
    b.check(b.run(num_sms=num_sms))


def test_long_context_and_growing_scores():
    """One long request (many pieces, many steps), with keys late in it whose scores exceed the earlier ones by far
    more than 2^8, so that the accumulators are rescaled."""
    b = Batch(_own([9000]), 8, 2, 128, seed=5)
    rng = np.random.default_rng(6)
    big = fp4.pack(*fp4.quantise(30 * rng.standard_normal((40, 2, 128)).astype(np.float32), KS))
    b.kp[b.table[0, 4000::130][:39]] = big[:39]
    b.check(b.run())
    # the same through tiles: a prefix that many requests share
    b = Batch(_star(40, 1200, 1, 9), 8, 1, 128, seed=7)
    b.kp[b.table[0, 600:1200:50]] = fp4.pack(*fp4.quantise(30 * rng.standard_normal((12, 1, 128)).astype(np.float32), KS))
    out = b.run()
    assert b.info["num_wide_items"] > 0
    b.check(out)


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (64, 8, 64), (8, 1, 128), (12, 12, 64)])
@pytest.mark.parametrize("n", [1, 170, 330])
def test_requests_of_one_piece(hq, hkv, d, n):
    """Short requests are not cut: the streams write their results, empty requests' among them, without a merge; with
    lengths that grow past the planned ones, in a graph, over poisoned partial rows."""
    rng = np.random.default_rng(n + d)
    lens = rng.integers(1, 40, n)
    lens[1::7] = 0
    b = Batch(_own(lens), hq, hkv, d, seed=n, extra=40)
    plan = b.plan()
    assert sgl.sgl_plan_info(plan)["num_merge_entries"] == b.B * hkv
    ws = torch.full((plan.workspace_bytes,), 0xFF, dtype=torch.uint8, device="cuda")
    ws[:256] = 0
    sgl.sgl_plan_upload(plan, ws)
    at = 0
    for r in range(n):                       # slots for the tokens to come
        grow = int(rng.integers(0, 40))
        take = b.free[at:at + grow]
        at += len(take)
        b.table[r, lens[r]:lens[r] + len(take)] = take
        lens[r] += len(take)
    new = b.table[b.table >= 0]
    for pool, s, i in ((b.kp, KS, 3), (b.vp, VS, 4)):
        pool[new] = _pool(b.slots, hkv, d, s, n + i)[new]
    kp, vp, t, dl = b.device()
    q = b.q.cuda()
    o = torch.full((n, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n, hq), 7.0, device="cuda")
    sgl.sgl_decode_attn(q, kp, vp, t, dl, plan, o, lse, ws)
    sgl.sgl_check(ws)
    rows = rng.permutation(n)[:16]
    b.check((o.double().cpu().numpy(), lse.double().cpu().numpy()), rows)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(2):
            sgl.sgl_decode_attn(q, kp, vp, t, dl, plan, o, lse, ws)
    o.fill_(7.0)
    lse.fill_(7.0)
    b.lens[:] = lens
    dl.copy_(torch.from_numpy(b.lens))
    g.replay()
    sgl.sgl_check(ws)
    b.check((o.double().cpu().numpy(), lse.double().cpu().numpy()), rows)


def test_offsets_past_32_bits():
    """Slots whose rows lie more than 2^31 bytes into the pools give what the same rows give in small pools, bit for
    bit: streams, tiles, extend and append."""
    hq, hkv, d = 32, 8, 128
    b = Batch(_star(20, 200, 1, 40), hq, hkv, d, seed=21)
    far = 2 ** 31 // sgl.sgl_fp4_row_bytes(hkv, d) + 1000
    rng = np.random.default_rng(22)
    pre = b.lens // 2
    ext = b.lens - pre
    n = int(ext.sum())
    q = torch.from_numpy(rng.standard_normal((n, hq, d)).astype(np.float32)).bfloat16().cuda()
    new = [torch.from_numpy(rng.standard_normal((b.B, hkv, d)).astype(np.float32)).bfloat16().cuda() for _ in "kv"]
    got = []
    for shift in (0, far):
        slots = b.slots + shift
        pools = []
        for x in (b.kp, b.vp):
            p = torch.zeros(slots, x.shape[1], dtype=torch.uint8, device="cuda")
            p[shift:] = torch.from_numpy(x).cuda()
            pools.append(p)
        table = torch.from_numpy(b.table + shift * (b.table >= 0)).int().cuda()
        lens, pd, ed = (torch.from_numpy(x.astype(np.int32)).cuda() for x in (b.lens, pre, ext))
        g = sgl.sgl_groups_create()
        sgl.sgl_groups_from_table(b.table, b.lens, g)
        mk = lambda **kw: sgl.make_params(sgl.SGL_DTYPE_BF16_FP4KV, b.B, hq, hkv, d, slots, k_scale=KS, v_scale=VS, **kw)  # noqa: E731
        plan = sgl.sgl_decode_plan(mk(), b.lens, sgl.sgl_groups_view(g))
        assert sgl.sgl_plan_info(plan)["num_wide_items"] > 0
        ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
        sgl.sgl_plan_upload(plan, ws)
        o, lse = torch.zeros(b.B, hq, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(b.B, hq, device="cuda")
        sgl.sgl_decode_attn(b.q.cuda(), *pools, table, lens, plan, o, lse, ws)
        p = mk(host_prefix_lens=pre, host_extend_lens=ext)
        oe, le = torch.zeros_like(q), torch.zeros(n, hq, device="cuda")
        sgl.sgl_extend_attn(q, *pools, table, pd, ed, p, oe, le, ws)
        sgl.sgl_kv_append(None, mk(), None, *new, *pools, table, lens, None, None, ws)
        sgl.sgl_check(ws)
        got.append([o, lse, oe, le] + [x[shift:].clone() for x in pools])
        sgl.sgl_groups_destroy(g)
        del pools
    for x, y in zip(*got):
        assert torch.equal(x, y)
    b.check((got[0][0].double().cpu().numpy(), got[0][1].double().cpu().numpy()))


def test_slots_outside_the_pool_are_skipped_and_reported():
    b = Batch(_own([100, 77, 5]), 32, 8, 128, seed=8)
    bad = b.table.copy()
    bad[0, 40], bad[0, 97], bad[1, 0], bad[1, 1], bad[1, 2], bad[1, 3] = b.slots, -5, 1 << 30, b.slots, -1, b.slots
    o, lse, ws = b.run(check=False, table=bad)
    with pytest.raises(sgl.SglError) as e:
        sgl.sgl_check(ws)
    assert e.value.status == -5
    for r, skip in enumerate(((40, 97), (0, 1, 2, 3), ())):
        _close(o[r], lse[r], b.ref(r, skip=skip))
    # a request all of whose slots are outside has nothing to attend to
    bad[2, :5] = b.slots
    o, lse, ws = b.run(check=False, table=bad)
    with pytest.raises(sgl.SglError):
        sgl.sgl_check(ws)
    assert (o[2] == 0).all() and np.isneginf(lse[2]).all()
    # a plan made for longer contexts than the device's lengths (a length is
    # seen to be too short where it lies before a piece that the plan made:
    # here the request's last piece, which starts at 32)
    plan = b.plan()
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    sgl.sgl_plan_upload(plan, ws)
    kp, vp, t, lens = b.device()
    out = torch.zeros(3, 32, 128, dtype=torch.bfloat16, device="cuda")
    lens[1] = 10
    sgl.sgl_decode_attn(b.q.cuda(), kp, vp, t, lens, plan, out, torch.zeros(3, 32, device="cuda"), ws)
    with pytest.raises(sgl.SglError):
        sgl.sgl_check(ws)


def test_nan_and_infinite_scales_reach_only_their_own_rows():
    b = Batch(_own([60, 60]), 16, 4, 64, seed=9)
    _, sf = fp4.unpack(b.vp, 4, 64)
    c, _ = fp4.unpack(b.vp, 4, 64)
    sf[b.table[0, 33], 2, 1] = 0x7F
    b.vp = fp4.pack(c, sf)
    o, lse = b.run()
    _close(o[1], lse[1], b.ref(1))
    hit = np.zeros((16, 64), dtype=bool)
    hit[8:12, 16:32] = True
    assert np.isnan(o[0][hit]).all() and not np.isnan(o[0][~hit]).any()


def test_query_outside_f16_is_reported():
    b = Batch(_own([60]), 8, 2, 128, seed=10)
    b.q[0, 3, 5] = 70000.0
    *_, ws = b.run(check=False)
    with pytest.raises(sgl.SglError):
        sgl.sgl_check(ws)


def test_decode_in_a_graph_and_on_two_streams():
    b = Batch(_star(12, 200, 1, 60) + EDGE, 32, 8, 128, seed=11)
    plan = b.plan()
    kp, vp, t, lens = b.device()
    q = b.q.cuda()
    work = []
    for i in range(2):
        s = torch.cuda.Stream()
        ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
        sgl.sgl_plan_upload(plan, ws)
        o, lse = torch.zeros_like(q), torch.zeros(b.B, 32, device="cuda")
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            sgl.sgl_decode_attn(q, kp, vp, t, lens, plan, o, lse, ws)
        work.append((s, ws, o, lse, g))
    for _ in range(5):
        for s, ws, o, lse, g in work:
            with torch.cuda.stream(s):
                o.zero_()
                g.replay()
    torch.cuda.synchronize()
    for s, ws, o, lse, g in work:
        sgl.sgl_check(ws)
        b.check((o.double().cpu().numpy(), lse.double().cpu().numpy()))
    assert torch.equal(work[0][2], work[1][2])


def test_no_alloc_decode():
    b = Batch(_star(5, 100, 1, 60), 32, 8, 128, seed=12)
    plan = b.plan()
    kp, vp, t, lens = b.device()
    o, lse = torch.zeros(5, 32, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(5, 32, device="cuda")
    sgl.sgl_decode_attn_noalloc(b.q.cuda(), kp, vp, t, lens, plan, o, lse)
    torch.cuda.synchronize()
    b.check((o.double().cpu().numpy(), lse.double().cpu().numpy()))


@pytest.mark.parametrize("shared", [False, True])
def test_decode_step_from_host_memory(shared):
    """One call from host memory (copies, decode with and without a merge, copies back) gives the separate calls'
    bytes."""
    b = Batch(_star(20, 200, 1, 30) if shared else _own([30, 0, 7, 50]), 32, 8, 128, seed=31)
    plan = b.plan()
    kp, vp, table, lens = b.device()
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    sgl.sgl_plan_upload(plan, ws)
    parts = [b.q, torch.from_numpy(b.table), torch.from_numpy(b.lens)]
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    at, spans = 0, []
    for x in parts:
        spans.append((at, x.numel() * x.element_size()))
        at += up(spans[-1][1])
    hin = torch.zeros(at, dtype=torch.uint8).pin_memory()
    for x, (o0, n) in zip(parts, spans):
        hin[o0:o0 + n] = x.reshape(-1).view(torch.uint8)
    din = torch.zeros(at, dtype=torch.uint8, device="cuda")
    q, t, sl = (din[o0:o0 + n].view(x.dtype).view(x.shape) for x, (o0, n) in zip(parts, spans))
    ob = up(b.q.numel() * 2)
    dout = torch.zeros(ob + b.B * b.hq * 4, dtype=torch.uint8, device="cuda")
    hout = torch.zeros(dout.numel(), dtype=torch.uint8).pin_memory()
    o = dout[:b.q.numel() * 2].view(torch.bfloat16).view(b.q.shape)
    lse = dout[ob:].view(torch.float32).view(b.B, b.hq)
    sgl.sgl_decode_step(hin, din, q, kp, vp, t, sl, plan, o, lse, dout, hout, ws)
    torch.cuda.synchronize()
    sgl.sgl_check(ws)
    o2, lse2 = torch.zeros_like(o), torch.zeros_like(lse)
    sgl.sgl_decode_attn(b.q.cuda(), kp, vp, table, lens, plan, o2, lse2, ws)
    assert torch.equal(hout[:b.q.numel() * 2], o2.reshape(-1).view(torch.uint8).cpu())
    assert torch.equal(hout[ob:], lse2.reshape(-1).view(torch.uint8).cpu())
    b.check((o2.double().cpu().numpy(), lse2.double().cpu().numpy()))


def test_refusals():
    from ctypes import byref
    b = Batch(_own([4]), 8, 2, 128)
    for kw, st in ((dict(k_scale=0.0), -1), (dict(v_scale=float("nan")), -1), (dict(k_scale=float("inf")), -1)):
        p = sgl.make_params(sgl.SGL_DTYPE_BF16_FP4KV, 1, 8, 2, 128, 100, **dict(dict(k_scale=1.0, v_scale=1.0), **kw))
        with pytest.raises(sgl.SglError) as e:
            sgl.sgl_extend_workspace_bytes(p)
        assert e.value.status == st
    plan = b.plan()
    lib = sgl._lib()
    assert lib.sgl_decode_attn(0x1000, 0x2008, 0x3000, 0x4000, 64, 0x5000, plan.handle, 0x6000, 0x7000, 0x8000, 1 << 30,
                               None) == -1
    assert lib.sgl_decode_attn(0x1000, 0x2000, 0x3000, 0x4000, 2, 0x5000, plan.handle, 0x6000, 0x7000, 0x8000, 1 << 30,
                               None) == -1
    assert lib.sgl_extend_attn(0x1000, 0x2000, None, 0x4000, 64, 0x5000, 0x5000,
                               byref(b.params(host_prefix_lens=[0], host_extend_lens=[4])), 0x6000, 0x7000, 0x8000,
                               256, None) == -1


# ------------------------------------------------------------------ extend
def _extend(b, pre, ext, q, write=None, rope=None, kp=None, vp=None):
    p = b.params(host_prefix_lens=pre, host_extend_lens=ext)
    kpd, vpd, t, _ = b.device()
    kpd = kpd if kp is None else kp
    vpd = vpd if vp is None else vp
    ws = torch.zeros(sgl.sgl_extend_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    pd, ed = (torch.from_numpy(np.asarray(x, dtype=np.int32)).cuda() for x in (pre, ext))
    o = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    if write is None:
        sgl.sgl_extend_attn(q.cuda(), kpd, vpd, t, pd, ed, p, o, lse, ws)
    else:
        sgl.sgl_extend_attn_kvwrite(q.cuda(), write[0].cuda(), write[1].cuda(), kpd, vpd, t, pd, ed, p, o, lse, ws)
    sgl.sgl_check(ws)
    return o.double().cpu().numpy(), lse.double().cpu().numpy(), kpd.cpu().numpy(), vpd.cpu().numpy()


def _check_extend(b, out, pre, ext, q, rows=None, **kw):
    at = 0
    for r in range(b.B):
        for i in range(int(ext[r])):
            if rows is None or at in rows:
                _close(out[0][at], out[1][at], b.ref(r, q=q[at], length=int(pre[r]) + i + 1, **kw))
            at += 1


@pytest.mark.parametrize("hq,hkv,d", [(64, 8, 128), (8, 8, 64), (16, 2, 64), (8, 1, 128), (10, 5, 64), (36, 9, 128)])
@pytest.mark.parametrize("fused", [False, True])
def test_extend(hq, hkv, d, fused):
    pre, ext = np.array([0, 150, 3, 60, 0]), np.array([70, 33, 1, 0, 140])
    b = Batch(_own(list(pre + ext)), hq, hkv, d, seed=hq)
    rng = np.random.default_rng(hq + 1)
    n = int(ext.sum())
    q = torch.from_numpy(rng.standard_normal((n, hq, d)).astype(np.float32)).bfloat16()
    write = None
    if fused:
        write = [torch.from_numpy(rng.standard_normal((n, hkv, d)).astype(np.float32)).bfloat16() for _ in "kv"]
        to = np.concatenate([b.table[r, pre[r]:pre[r] + ext[r]] for r in range(b.B)])
        want = []
        for pool, x, s in ((b.kp, write[0], KS), (b.vp, write[1], VS)):
            w = pool.copy()
            rows = fp4.pack(*fp4.quantise(x.float().numpy(), s))
            used = hkv * (d // 2 + d // 16)
            w[to, :used] = rows[:, :used]
            want.append(w)
            pool[to, :used] = 0xFF                 # what was there before
    out = _extend(b, pre, ext, q, write)
    if fused:
        assert np.array_equal(out[2], want[0]) and np.array_equal(out[3], want[1])
        b.kp, b.vp = want
    _check_extend(b, out, pre, ext, q)


def test_extend_long_prefix():
    pre, ext = np.array([2111, 4000]), np.array([300, 129])
    b = Batch(_own(list(pre + ext)), 32, 4, 128, page=16, seed=13)
    rng = np.random.default_rng(14)
    q = torch.from_numpy(rng.standard_normal((int(ext.sum()), 32, 128)).astype(np.float32)).bfloat16()
    out = _extend(b, pre, ext, q)
    _check_extend(b, out, pre, ext, q, rows={0, 1, 15, 16, 31, 32, 127, 128, 299, 300, 331, 428})


# ------------------------------------------------------------------ a run of them
@pytest.mark.parametrize("hq,hkv,d,page", [(32, 8, 128, 16), (16, 2, 64, 1)])
def test_prefill_then_decode_steps(hq, hkv, d, page):
    """As a serving loop uses them: prompts are rotated and appended in chunks and attended, then every request decodes
    token by token (append, then decode over a plan that is reused as the batch grows), in a graph per plan."""
    rng = np.random.default_rng(hq)
    prompt = np.array([40, 0, 97, 16, 200])
    B, steps = len(prompt), 37
    b = Batch(_own(list(prompt + steps)), hq, hkv, d, page=page, seed=15)
    b.kp[:], b.vp[:] = 0xFF, 0xFF
    total = b.lens.copy()
    freq = orope.frequencies(d, 10000.0, "yarn", factor=4.0, original=64, low=1.0, high=32.0)
    amp = 0.1 * np.log(4.0) + 1.0
    rope = sgl.sgl_rope_create(d, scaling=sgl.SGL_ROPE_SCALE_YARN, factor=4.0, original_positions=64, low=1.0, high=32.0)
    kp, vp, table, _ = b.device()
    draw = lambda n, h: torch.from_numpy(rng.standard_normal((n, h, d)).astype(np.float32)).bfloat16()  # noqa: E731

    def book(qr, x_k, x_v, rows):
        """The oracle's pools after the rows (request, position) were appended; the rotated query is the library's (its
        rotation has a test of its own), the key's is checked here through its codes."""
        for i, (r, p) in enumerate(rows):
            k = orope.rotate(x_k[i].double().numpy()[None], [p], freq, amplitude=amp)[0]
            k = torch.from_numpy(k).float().bfloat16().float().numpy()
            for pool, host, x, s in ((kp, b.kp, k, KS), (vp, b.vp, x_v[i].float().numpy(), VS)):
                slot = b.table[r, p]
                want = fp4.pack(*fp4.quantise(x[None], s))[0]
                got = pool[slot].cpu().numpy()
                used = hkv * (d // 2 + d // 16)
                # (a rotated key may round the other way at a border: hardly any code differs, by one step)
                assert np.mean(got[:used] != want[:used]) < 0.05
                host[slot] = got

    # prompts, in two chunks
    done = np.zeros(B, dtype=np.int64)
    for part in (prompt // 2, prompt - prompt // 2):
        rows = [(r, int(done[r]) + i) for r in range(B) for i in range(part[r])]
        n = len(rows)
        q, k, v = draw(n, hq), draw(n, hkv), draw(n, hkv)
        p = b.params(host_prefix_lens=done, host_extend_lens=part)
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        pre, ext = (torch.from_numpy(x.astype(np.int32)).cuda() for x in (done, part))
        qr = torch.zeros(n, hq, d, dtype=torch.bfloat16, device="cuda")
        o, lse = torch.zeros_like(qr), torch.zeros(n, hq, device="cuda")
        sgl.sgl_kv_append(rope, p, q.cuda(), k.cuda(), v.cuda(), kp, vp, table, pre, ext, qr, ws)
        sgl.sgl_extend_attn(qr, kp, vp, table, pre, ext, p, o, lse, ws)
        sgl.sgl_check(ws)
        book(qr, k, v, rows)
        _check_extend(b, (o.double().cpu().numpy(), lse.double().cpu().numpy()), done, part, qr.cpu())
        done = done + part
    # decode steps: one plan for all of them, made for the lengths after the first append
    b.lens = (done + 1).astype(np.int32)
    plan = b.plan()
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    sgl.sgl_plan_upload(plan, ws)
    lens = torch.from_numpy(done.astype(np.int32)).cuda()
    qd, kd, vd = (torch.zeros(B, h, d, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv, hkv))
    qr, o, lse = torch.zeros_like(qd), torch.zeros_like(qd), torch.zeros(B, hq, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lens.add_(1)
        sgl.sgl_kv_append(rope, b.params(), qd, kd, vd, kp, vp, table, lens, None, qr, ws)
        sgl.sgl_decode_attn(qr, kp, vp, table, lens, plan, o, lse, ws)
    for step in range(steps):
        q, k, v = draw(B, hq), draw(B, hkv), draw(B, hkv)
        qd.copy_(q)
        kd.copy_(k)
        vd.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        sgl.sgl_check(ws)
        book(qr, k, v, [(r, int(done[r])) for r in range(B)])
        done = done + 1
        b.lens = done.astype(np.int32)
        for r in range(B):
            _close(o[r].double().cpu().numpy(), lse[r].double().cpu().numpy(), b.ref(r, q=qr[r].cpu()))
    assert np.array_equal(done, total)
