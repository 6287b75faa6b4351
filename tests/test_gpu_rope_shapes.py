"""The rotation and the append on both sides of every size at which the launch changes: below 152 rows a token's heads
are dealt to several CTAs, from 304 rows on two tokens share a CTA.

Rotated rows are held to the float64 rotation, appended ones to the bytes of the rows that `sgl_rope` gives.
"""

import numpy as np
import pytest
import torch

import radixattention_prefix_shared_radix_gb300 as sgl
from tests.test_rope import KINDS, _bytes, _check_rotated, _pool, _rope, _stored

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from radixattention_prefix_shared_radix_gb300 import build
    build.build()


@pytest.mark.parametrize("n", [151, 152, 153, 303, 304, 305, 611])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hq,hk,d,rot,off", [(3, 1, 64, 64, 0), (40, 9, 128, 64, 32), (5, 2, 80, 64, 16)])
def test_rotation_at_the_launch_shapes(n, dtype, hq, hk, d, rot, off):
    r, freq, amp = _rope(d, rot, off, False, "banded")
    g = torch.Generator().manual_seed(n)
    q = torch.randn(n, hq, d, generator=g).to(dtype).cuda()
    k = torch.randn(n, hk, d, generator=g).to(dtype).cuda()
    pos = torch.randint(0, 5000, (n,), generator=g, dtype=torch.int32)
    pos[n // 2] = -1
    qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    sgl.sgl_rope(r, q, k, pos.cuda(), qo, ko)
    p = pos.numpy().astype(np.int64)
    _check_rotated(qo, q, p, rot, off, False, freq, amp)
    _check_rotated(ko, k, p, rot, off, False, freq, amp)
    assert (qo[n // 2] == 7).all() and (ko[n // 2] == 7).all()


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("n", [151, 152, 153, 303, 304, 305, 611])
@pytest.mark.parametrize("decode", [False, True])
def test_append_at_the_launch_shapes(kind, n, decode):
    hq, hkv, d, rot = 10, 5, 64, 32
    rng = np.random.default_rng(n)
    B = n if decode else 4
    ext = np.ones(B, dtype=np.int64)
    if not decode:
        cut = np.sort(rng.integers(0, n - 6, 3))
        ext = np.diff(np.concatenate([[0], cut, [n - 7]]))       # (seven rows of padding)
    rows = int(ext.sum())
    pre = rng.integers(0, 40, B)
    ld, slots = int((pre + ext).max()) + 1, n + 9
    order = rng.permutation(slots)[:rows]
    table = np.full((B, ld), -1, dtype=np.int32)
    who = [(r, i) for r in range(B) for i in range(ext[r])]
    for at, (r, i) in enumerate(who):
        table[r, pre[r] + i] = order[at]
    dt = torch.float32 if kind == "f32" else torch.bfloat16
    g = torch.Generator().manual_seed(n)
    q, k, v = (torch.randn(n, h, d, generator=g).to(dt).cuda() for h in (hq, hkv, hkv))
    rope, freq, amp = _rope(d, rot)
    ks, vs = 0.37, 1.3
    params = sgl.make_params(KINDS[kind], B, hq, hkv, d, slots, k_scale=ks, v_scale=vs)
    kp, vp = _pool(kind, slots, hkv, d, 1), _pool(kind, slots, hkv, d, 2)
    kb, vb = _bytes(kp), _bytes(vp)
    qo = torch.full_like(q, 7.0)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    lens = torch.from_numpy((pre + 1 if decode else pre).astype(np.int32)).cuda()
    extd = None if decode else torch.from_numpy(ext.astype(np.int32)).cuda()
    sgl.sgl_kv_append(rope, params, q, k, v, kp, vp, torch.from_numpy(table).cuda(), lens, extd, qo, ws)
    sgl.sgl_check(ws)
    pos = np.array([pre[a] + i for a, i in who])
    _check_rotated(qo[:rows], q[:rows], pos, rot, 0, False, freq, amp)
    assert (qo[rows:] == 7).all()
    kr = torch.empty_like(k)
    sgl.sgl_rope(rope, None, k, torch.from_numpy(np.concatenate([pos, np.zeros(n - rows)]).astype(np.int32)).cuda(),
                 None, kr)
    kb[order] = _stored(kind, kr[:rows], ks, hkv, d, kb[order])
    vb[order] = _stored(kind, v[:rows], vs, hkv, d, vb[order])
    assert np.array_equal(_bytes(kp), kb) and np.array_equal(_bytes(vp), vb)
