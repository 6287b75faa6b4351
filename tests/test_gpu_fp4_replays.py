"""Decode steps over a 4-bit cache with a shared prefix (tiles, the streams behind them and the merge), captured once
with the append before them and replayed while inputs, lengths and the cache move on, nothing waited for in between."""

import numpy as np
import pytest
import torch

import radixattention_prefix_shared_radix_gb300 as sgl
from oracle import fp4
from tests.test_gpu_fp4 import KS, VS, Batch, _close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from radixattention_prefix_shared_radix_gb300 import build
    build.build()


@pytest.mark.parametrize("hq,hkv,d,prefix", [(32, 8, 128, 400), (16, 2, 64, 700), (32, 8, 128, 0)])
def test_steps_replayed_over_a_shared_prefix(hq, hkv, d, prefix):
    n, steps = 24, 30
    rng = np.random.default_rng(prefix)
    own = rng.integers(1, 60, n)
    b = Batch([([("p", prefix)] if prefix else []) + [(r, int(own[r]) + steps)] for r in range(n)], hq, hkv, d, seed=prefix)
    start = b.lens - steps
    # what is appended later holds NaN until then
    for r in range(n):
        for pool in (b.kp, b.vp):
            pool[b.table[r, start[r]:b.lens[r]]] = 0xFF
    first = (start + 1).astype(np.int32)
    g = sgl.sgl_groups_create()
    sgl.sgl_groups_from_table(b.table, first, g)
    plan = sgl.sgl_decode_plan(b.params(), first, sgl.sgl_groups_view(g))
    sgl.sgl_groups_destroy(g)
    assert (sgl.sgl_plan_info(plan)["num_wide_items"] > 0) == (prefix > 0)
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    sgl.sgl_plan_upload(plan, ws)
    kp, vp, table, _ = b.device()
    gen = torch.Generator().manual_seed(prefix)
    q, k, v = (torch.randn(steps, n, h, d, generator=gen).bfloat16().cuda() for h in (hq, hkv, hkv))
    rope = sgl.sgl_rope_create(d)
    lens = torch.from_numpy(start.astype(np.int32)).cuda()
    qd, kd, vd = (torch.zeros_like(x[0]) for x in (q, k, v))
    qr, o, lse = torch.zeros_like(qd), torch.zeros_like(qd), torch.zeros(n, hq, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lens.add_(1)
        sgl.sgl_kv_append(rope, b.params(), qd, kd, vd, kp, vp, table, lens, None, qr, ws)
        sgl.sgl_decode_attn(qr, kp, vp, table, lens, plan, o, lse, ws)
    outs = []
    for i in range(steps):
        qd.copy_(q[i])
        kd.copy_(k[i])
        vd.copy_(v[i])
        graph.replay()
        outs.append((qr.clone(), o.clone(), lse.clone()))
    sgl.sgl_check(ws)
    K, V = (fp4.Fp4View(x.cpu().numpy(), hkv, d, s) for x, s in ((kp, KS), (vp, VS)))
    for i, (qi, oi, li) in enumerate(outs):
        oi, li = oi.double().cpu().numpy(), li.double().cpu().numpy()
        for r in rng.permutation(n)[:6]:
            length = int(start[r]) + 1 + i
            _close(oi[r], li[r], b.ref(r, q=qi[r].cpu(), length=length, kp=K.rows, vp=V.rows))


@pytest.mark.parametrize("hq,hkv,d,prefix", [(32, 8, 128, 400), (16, 2, 64, 700), (32, 8, 128, 0)])
def test_steps_back_to_back_read_what_was_just_written(hq, hkv, d, prefix):
    """Append and decode again and again over one query buffer, one slot per request and one workspace, with no other
    kernel in between: each decode sees its own append, not the one before it.  Held to the same calls with a wait after
    each, bit for bit."""
    n, steps = 24, 12
    rng = np.random.default_rng(prefix + 1)
    b = Batch([([("p", prefix)] if prefix else []) + [(r, int(rng.integers(1, 200)))] for r in range(n)], hq, hkv, d,
              seed=prefix + 1)
    plan = b.plan()
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    sgl.sgl_plan_upload(plan, ws)
    kp, vp, table, lens = b.device()
    gen = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(steps, n, h, d, generator=gen).bfloat16().cuda() for h in (hq, hkv, hkv))
    rope = sgl.sgl_rope_create(d)
    qr = torch.zeros_like(q[0])

    def run(wait):
        o, lse = torch.zeros_like(q), torch.zeros(steps, n, hq, device="cuda")

        def calls():
            for i in range(steps):
                sgl.sgl_kv_append(rope, b.params(), q[i], k[i], v[i], kp, vp, table, lens, None, qr, ws)
                sgl.sgl_decode_attn(qr, kp, vp, table, lens, plan, o[i], lse[i], ws)
                if wait:
                    torch.cuda.synchronize()
        if wait:
            calls()
            return o, lse
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            calls()
        for _ in range(10):
            o.zero_()
            graph.replay()
        torch.cuda.synchronize()
        return o, lse
    want = run(True)
    assert not any(torch.equal(want[0][i], want[0][i + 1]) for i in range(steps - 1))
    got = run(False)
    sgl.sgl_check(ws)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # and outside a graph
    o, lse = torch.zeros_like(q), torch.zeros(steps, n, hq, device="cuda")
    for i in range(steps):
        sgl.sgl_kv_append(rope, b.params(), q[i], k[i], v[i], kp, vp, table, lens, None, qr, ws)
        sgl.sgl_decode_attn(qr, kp, vp, table, lens, plan, o[i], lse[i], ws)
    sgl.sgl_check(ws)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
