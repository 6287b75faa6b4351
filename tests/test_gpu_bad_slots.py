"""Slots outside the pool in the tiles of shared prefixes and in extend, over 4-bit pools: nothing is read for them (the
position counts as a zero key and a zero value) and they are reported, in a pool without any rows too."""

import numpy as np
import pytest
import torch

import radixattention_prefix_shared_radix_gb300 as sgl
from oracle import fp4
from tests.test_gpu_fp4 import KS, VS, _own, _ref, _star
from tests.test_gpu_nan import Run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from radixattention_prefix_shared_radix_gb300 import build
    build.build()


def _values(r, pool, scale, slots, bad):
    """Float64 rows of `slots`, zeros where `bad`."""
    return np.where(bad[:, None, None], 0.0, fp4.values(pool.numpy()[np.where(bad, 0, slots)], r.hkv, r.d, scale))


def _check(r, table, slots_in_pool, o, lse, q, req, length):
    slots = table[req, :length]
    bad = (slots < 0) | (slots >= slots_in_pool)
    O, L, to, tl = _ref(q.double().numpy(), _values(r, r.k, KS, slots, bad), _values(r, r.v, VS, slots, bad),
                        1 / np.sqrt(r.d))
    assert (np.abs(o.double().numpy() - O) <= to).all() and (np.abs(lse.double().numpy() - L) <= tl).all()


@pytest.mark.parametrize("hq,hkv,d", [(16, 4, 64), (32, 8, 128), (9, 9, 64)])
@pytest.mark.parametrize("rows", [None, 0])
def test_extend(hq, hkv, d, rows):
    pre, ext = np.array([0, 150, 30]), np.array([140, 70, 1])
    r = Run("fp4", _own(list(pre + ext)), hq, hkv, d, seed=11)
    b, n = r.b, int(ext.sum())
    slots = b.slots if rows is None else rows
    b.table[0, 7], b.table[0, 100], b.table[1, 20], b.table[1, 199], b.table[2, 30] = slots, -1, 1 << 30, -7, slots
    b.slots = slots
    q = torch.randn(n, hq, d, generator=torch.Generator().manual_seed(1)).bfloat16()
    p = r.params(host_prefix_lens=pre, host_extend_lens=ext)
    ws = torch.zeros(sgl.sgl_extend_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    pd, ed = (torch.from_numpy(x.astype(np.int32)).cuda() for x in (pre, ext))
    o, lse = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda"), torch.full(q.shape[:2], 7.0, device="cuda")
    sgl.sgl_extend_attn(q.cuda(), r.k.cuda(), r.v.cuda(), torch.from_numpy(b.table).cuda(), pd, ed, p, o, lse, ws)
    with pytest.raises(sgl.SglError) as e:
        sgl.sgl_check(ws)
    assert e.value.status == -5
    o, lse, at = o.cpu(), lse.cpu(), 0
    for req in range(3):
        for i in range(ext[req]):
            _check(r, b.table, slots, o[at], lse[at], q[at], req, int(pre[req]) + i + 1)
            at += 1


@pytest.mark.parametrize("hq,hkv,d", [(16, 4, 64), (32, 8, 128)])
def test_shared_prefix(hq, hkv, d):
    # (own parts of one token: what is read for the tiles is the prefix alone)
    r = Run("fp4", _star(30, 500, 1, 1), hq, hkv, d, seed=12)
    b = r.b
    g = sgl.sgl_groups_create()
    sgl.sgl_groups_from_table(b.table, b.lens, g)
    plan = sgl.sgl_decode_plan(r.params(), b.lens, sgl.sgl_groups_view(g))
    sgl.sgl_groups_destroy(g)
    assert sgl.sgl_plan_info(plan)["num_wide_items"] > 0
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    sgl.sgl_plan_upload(plan, ws)
    b.table[:, 3], b.table[:, 130], b.table[:, 499] = b.slots, -1, 1 << 30
    q = r.q.cuda()
    o, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    sgl.sgl_decode_attn(q, r.k.cuda(), r.v.cuda(), torch.from_numpy(b.table).cuda(), torch.from_numpy(b.lens).cuda(), plan,
                        o, lse, ws)
    with pytest.raises(sgl.SglError) as e:
        sgl.sgl_check(ws)
    assert e.value.status == -5
    o, lse = o.cpu(), lse.cpu()
    for req in range(b.B):
        _check(r, b.table, b.slots, o[req], lse[req], r.q[req], req, int(b.lens[req]))
