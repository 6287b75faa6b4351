"""Rows from sgl_build_batch that share a prefix, are thinned out by the attention that their tokens get, grow by
sgl_batch_append and end: attention outputs, log-sum-exps, scores and rotations against float64 over the pools' contents,
selections against the oracle's, and every page of the tree accounted for."""

import numpy as np
import pytest
import torch

import radixattention_prefix_shared_radix_gb300 as sgl
from oracle import evict as oevict, fp4
from oracle.fp8 import e4m3_to_float
from tests.test_gpu_attn_weights import KINDS, Cache
from tests.test_gpu_fp4 import KS, VS
from tests.test_rope_axes import _axes, _check

pytestmark = pytest.mark.gpu

HQ, HKV, D, SLOTS, LD = 8, 2, 64, 768, 192
AXES = (12, 10, 10)


@pytest.fixture(scope="module", autouse=True)
def _built():
    from radixattention_prefix_shared_radix_gb300 import build
    build.build()


def _values(kind, pool, rows, scale):
    x = pool[torch.from_numpy(rows.astype(np.int64)).cuda()].cpu()
    if kind == "fp4":
        c, s = fp4.unpack(x.numpy(), HKV, D)
        return scale * fp4.e2m1_to_float(c) * np.repeat(e4m3_to_float(s), 16, -1)
    if kind == "fp8":
        return scale * e4m3_to_float(x.numpy())
    return x.double().numpy()


def _hold_attention(kind, q, kp, vp, table, pre, ext, o, lse):
    """Rows in request order, row i of request r at position pre[r] + i.  A score is off as in oracle/evict.py: by
    rel = (size (d + 12) + |score|) 2^-24 + (sum |k|) 2^-25 and a few roundings of 2^-21; a weight by rel of itself and,
    rounded for the second product, by half a step (bf16 2^-8, f16 2^-11); the weights' sum by rel; the output by half
    a step of its own."""
    q, o, lse = (x.double().cpu().numpy() for x in (q, o, lse))
    half_p = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}.get(kind, 2.0 ** -11)
    half_o = 2.0 ** -24 if kind == "f32" else 2.0 ** -8
    at = 0
    for r in range(len(pre)):
        n, L = int(ext[r]), int(pre[r] + ext[r])
        k, v = (_values(kind, p, table[r, :L], s) for p, s in ((kp, KS), (vp, VS)))
        for h in range(HQ):
            kh, vh, x = k[:, h * HKV // HQ], v[:, h * HKV // HQ], q[at:at + n, h]
            s = x @ kh.T / 8
            s[np.arange(L)[None] > pre[r] + np.arange(n)[:, None]] = -np.inf
            top = s.max(1, keepdims=True)
            w = np.exp(s - top)
            total = w.sum(1, keepdims=True)
            w /= total
            size = np.abs(x) @ np.abs(kh).T / 8
            rel = ((size * (D + 12) + np.abs(np.where(w > 0, s, 0)) + np.abs(top)) * 2.0 ** -24
                   + np.abs(kh).sum(1) / 8 * 2.0 ** -25 + 2.0 ** -20).max(1, keepdims=True)
            ref, spread = w @ vh, w @ np.abs(vh)
            assert (np.abs(o[at:at + n, h] - ref) <= spread * (half_p + 2 * rel) * 1.01 + np.abs(ref) * half_o).all()
            want = (top + np.log(total))[:, 0]
            assert (np.abs(lse[at:at + n, h] - want) <= rel[:, 0] + (np.abs(want) + 1) * 2.0 ** -22).all()
        at += n


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("P", [1, 16])
def test_thinned_rows_of_a_batch(kind, P):
    g = torch.Generator().manual_seed(12)
    rng = np.random.default_rng(5)
    prompts = [np.concatenate([np.arange(48), 1000 * r + np.arange(n)]).astype(np.int32)
               for r, n in enumerate((37, 64, 5, 100), 1)]
    B = len(prompts)
    tree = sgl.sgl_tree_create(SLOTS, P, rng.permutation(SLOTS // P).astype(np.int32))
    out = sgl.sgl_build_batch(tree, prompts, ld=LD)
    row, lens, pre = out["req_to_token"], out["seq_lens"], out["prefix_lens"].astype(np.int64)
    n0 = lens.astype(np.int64)
    assert pre.tolist() == [0, 48, 48, 48]
    first = row.copy()
    nodes = [set(row[r, :n0[r] // P * P].tolist()) for r in range(B)]
    own = [set(row[r, n0[r] // P * P:n0[r]].tolist()) for r in range(B)]
    held = sgl.sgl_tree_stats(tree)["tree_tokens"]
    dt = torch.float32 if kind == "f32" else torch.bfloat16
    if kind == "fp4":
        kp, vp = (torch.full((SLOTS, fp4.row_bytes(HKV, D)), 0xFF, dtype=torch.uint8, device="cuda") for _ in "kv")
    elif kind == "fp8":
        kp, vp = (torch.full((SLOTS, HKV, D), 0x7F, dtype=torch.uint8, device="cuda") for _ in "kv")
    else:
        kp, vp = (torch.full((SLOTS, HKV, D), float("nan"), dtype=dt, device="cuda") for _ in "kv")
    rope, freq, axis, amp = _axes(D, D, AXES)
    c = Cache(kind, [0] * B, HQ, HKV, D, ld=LD, seed=11)
    c.slots = SLOTS
    td, ld_ = torch.from_numpy(row).cuda(), torch.from_numpy(lens).cuda()
    scores = torch.zeros(B, LD, device="cuda")
    posr = torch.arange(LD, dtype=torch.int32, device="cuda").repeat(B, 1)
    budget, recent = [40, 64, 60, 48], 6
    bud = torch.tensor(budget, dtype=torch.int32, device="cuda")
    ev, cnt = torch.zeros(B, LD, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")

    def places(i):          # a token's on each axis; the shared ones' are everybody's
        return torch.stack([i, (3 * i) % 11 + 2, (5 * i) % 23]).to(torch.int32)

    def new(n):
        return [torch.randn(n, h, D, generator=g).to(dt).cuda() for h in (HQ, HKV, HKV)]

    def hold(pre, ext, q, turned, at, o, lse, before, window, decode):
        _check(turned, q, at.numpy().astype(np.int64), D, 0, False, freq, axis, amp)
        c.table, c.pool = td.cpu().numpy(), kp.cpu()
        _hold_attention(kind, turned, kp, vp, c.table, pre, ext, o, lse)
        want, tol = c.expect(turned.cpu(), lse.cpu(), pre, ext, window, before, 1.0, decode, 0.125)
        live = np.arange(LD)[None] < (pre + ext)[:, None]
        assert (np.abs(scores.cpu().numpy() - want) <= tol)[live].all()

    def thin(ws):
        was = [x.cpu().numpy().copy() for x in (scores, td, posr, ld_)]
        sgl.sgl_kv_evict(scores, td, ld_, bud, scores, td, ld_, ws, ev, cnt, posr, posr, page_size=P, sinks=2, recent=recent)
        sgl.sgl_check(ws)
        for r in range(B):
            n = int(was[3][r])
            stays = oevict.keep(was[0][r, :n], budget[r], P, 2, recent)
            m = int(stays.sum())
            assert int(ld_[r]) == m
            for x, y in ((scores, was[0]), (td, was[1]), (posr, was[2])):
                assert np.array_equal(x[r, :m].cpu().numpy(), y[r, :n][stays])
            gone = ev[r, :int(cnt[r])].cpu().numpy()
            assert np.array_equal(gone, was[1][r, :n][~stays])
            mine = [s for s in gone.tolist() if s not in nodes[r]]
            assert own[r].issuperset(mine) and len(mine) % P == 0
            own[r].difference_update(mine)
            if mine:
                sgl.sgl_tree_free(tree, np.array(mine, dtype=np.int32))

    # prompts
    ext = n0 - pre
    index = torch.cat([torch.arange(int(a), int(b)) for a, b in zip(pre, n0)])
    q, k, v = new(int(ext.sum()))
    p = c.params(host_prefix_lens=pre, host_extend_lens=ext)
    ws = torch.zeros(max(sgl.sgl_extend_workspace_bytes(p), sgl.sgl_attn_weights_workspace_bytes(p, 8)), dtype=torch.uint8,
                     device="cuda")
    pd, ed = (torch.from_numpy(x.astype(np.int32)).cuda() for x in (pre, ext))
    turned, o, lse = torch.empty_like(q), torch.empty_like(q), torch.empty(len(q), HQ, device="cuda")
    sgl.sgl_kv_append_at(rope, p, q, k, v, kp, vp, td, pd, ed, places(index).cuda(), turned, ws)
    sgl.sgl_extend_attn(turned, kp, vp, td, pd, ed, p, o, lse, ws)
    sgl.sgl_attn_weights(turned, lse, kp, td, pd, ed, p, None, scores, ws, window=8)
    sgl.sgl_check(ws)
    hold(pre, ext, q, turned, places(index), o, lse, np.zeros((B, LD), dtype=np.float32), 8, False)
    thin(ws)
    # steps: rows that no longer count their tokens
    for step in range(6):
        host, seq = td.cpu().numpy(), ld_.cpu().numpy()
        had = seq.astype(np.int64)
        sgl.sgl_batch_append(tree, host, seq)
        for r in range(B):
            s = int(host[r, had[r]])
            assert s not in own[r] and s not in set().union(*nodes) and not any(s in x for x in own)
            own[r].add(s)
            posr[r, int(had[r])] = int(n0[r]) + step
        td.copy_(torch.from_numpy(host))
        ld_.copy_(torch.from_numpy(seq))
        q, k, v = new(B)
        at = places(torch.from_numpy(n0) + step)
        turned, o, lse = torch.empty_like(q), torch.empty_like(q), torch.empty(B, HQ, device="cuda")
        grp = sgl.sgl_groups_create()
        sgl.sgl_groups_from_table(host, seq, grp)
        pd = c.params()
        plan = sgl.sgl_decode_plan(pd, seq, sgl.sgl_groups_view(grp))
        sgl.sgl_groups_destroy(grp)
        wd = torch.zeros(max(256, plan.workspace_bytes), dtype=torch.uint8, device="cuda")
        sgl.sgl_plan_upload(plan, wd)
        before = scores.cpu().numpy().copy()
        sgl.sgl_kv_append_at(rope, pd, q, k, v, kp, vp, td, ld_, None, at.cuda(), turned, wd)
        sgl.sgl_decode_attn(turned, kp, vp, td, ld_, plan, o, lse, wd)
        sgl.sgl_attn_weights(turned, lse, kp, td, ld_, None, pd, scores, scores, wd)
        sgl.sgl_check(wd)
        hold(had, np.ones(B, dtype=np.int64), q, turned, at, o, lse, before, 0, True)
        thin(wd)
    # their ends: all pages are free or cached, and the prompts' full pages still are
    for r in range(B):
        sgl.sgl_tree_unlock(tree, int(out["last_nodes"][r]))
        if own[r]:
            sgl.sgl_tree_free(tree, np.array(sorted(own[r]), dtype=np.int32))
    st = sgl.sgl_tree_stats(tree)
    assert st["locked_tokens"] == 0 and st["tree_tokens"] == held and st["free_pages"] * P + held == SLOTS
    for r in range(B):
        m, slots, _ = sgl.sgl_tree_match(tree, prompts[r])
        assert m == n0[r] // P * P and np.array_equal(slots, first[r, :m])
    sgl.sgl_tree_destroy(tree)
