"""Rows that an append at positions leaves out (a negative position on some axis): their slots and lengths may be
anything inside the table, and nothing is reported for them."""

import numpy as np
import pytest
import torch

import radixattention_prefix_shared_radix_gb300 as sgl
from tests.test_rope import KINDS, _bytes, _pool

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from radixattention_prefix_shared_radix_gb300 import build
    build.build()


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("axes", [(64,), (16, 24, 24)])
@pytest.mark.parametrize("decode", [False, True])
def test_nothing_is_reported_for_rows_left_out(kind, axes, decode):
    B, hq, hkv, d, slots, ld = 5, 4, 2, 128, 64, 16
    g = torch.Generator().manual_seed(1)
    dt = torch.float32 if kind == "f32" else torch.bfloat16
    q, k, v = (torch.randn(B, h, d, generator=g).to(dt).cuda() for h in (hq, hkv, hkv))
    rope = sgl.sgl_rope_create(d, axes=axes)
    p = sgl.make_params(KINDS[kind], B, hq, hkv, d, slots, k_scale=0.37, v_scale=1.3)
    table = np.full((B, ld), -1, dtype=np.int32)
    # rows 0 and 3 are appended; 1: no slot; 2: a slot behind the pool; 4: past the table
    table[0, 4], table[3, 2], table[2, 7] = 11, 12, slots
    lens = np.array([5, 3, 8, 3, ld + 1], dtype=np.int32) - (0 if decode else 1)
    pos = torch.randint(0, 9000, (len(axes), B), generator=g, dtype=torch.int32)
    left = [1, 2, 4]
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    td, ld_ = torch.from_numpy(table).cuda(), torch.from_numpy(lens).cuda()
    ext = None if decode else torch.ones(B, dtype=torch.int32, device="cuda")

    def append(rows):
        at = pos.clone()
        at[-1, rows] = -1
        kp, vp = _pool(kind, slots, hkv, d, 1), _pool(kind, slots, hkv, d, 2)
        before = [_bytes(x) for x in (kp, vp)]
        qo = torch.full_like(q, 7.0)
        sgl.sgl_kv_append_at(rope, p, q, k, v, kp, vp, td, ld_, ext, at.cuda(), qo, ws)
        return [(_bytes(x) != y).reshape(slots, -1).any(1) for x, y in zip((kp, vp), before)], qo

    changed, qo = append(left)
    sgl.sgl_check(ws)
    assert all(np.nonzero(x)[0].tolist() == [11, 12] for x in changed)
    assert (qo[left] == 7).all() and not (qo[[0, 3]] == 7).any()
    for r in left:                                 # each of them is reported when it takes part
        append([x for x in left if x != r])
        with pytest.raises(sgl.SglError) as e:
            sgl.sgl_check(ws)
        assert e.value.status == -5
