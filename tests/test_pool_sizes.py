"""Calls that write a pool refuse one that cannot hold its rows."""

import numpy as np
import pytest
import torch

import radixattention_prefix_shared_radix_gb300 as sgl
from oracle import fp4

KINDS = {sgl.SGL_DTYPE_F32: torch.float32, sgl.SGL_DTYPE_BF16: torch.bfloat16, sgl.SGL_DTYPE_BF16_FP8KV: torch.uint8}


@pytest.mark.parametrize("hkv,d", [(1, 64), (5, 64), (8, 128), (3, 128)])
def test_row_bytes(hkv, d):
    for kind in range(4):
        p = sgl.make_params(kind, 1, hkv, hkv, d, 10)
        want = fp4.row_bytes(hkv, d) if kind == sgl.SGL_DTYPE_BF16_FP4KV else hkv * d * KINDS[kind].itemsize
        assert sgl._row_bytes(p) == want


def test_a_pool_below_its_rows_is_refused():
    t = torch.zeros(10, 288, dtype=torch.uint8)
    assert sgl._writable(5, t, "k_pool", 2880) == 5 and sgl._writable(5, t, "k_pool", 0) == 5
    with pytest.raises(ValueError, match="v_pool must hold"):
        sgl._writable(5, t, "v_pool", 2881)


@pytest.mark.gpu
def test_writes_check_their_pools():
    """Refused before the library is called: nothing is written, whichever of the pools is too small."""
    B, hkv, d, slots = 2, 4, 64, 32
    row = sgl.sgl_fp4_row_bytes(hkv, d)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table, lens, zero = torch.arange(B * 4, device="cuda").int().view(B, 4), i32([1, 1]), i32([0, 0])
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    for kind in range(4):
        dt = torch.float32 if kind == sgl.SGL_DTYPE_F32 else torch.bfloat16
        p = sgl.make_params(kind, B, hkv, hkv, d, slots, host_prefix_lens=[0, 0], host_extend_lens=[1, 1])
        new = torch.ones(B, hkv, d, dtype=dt, device="cuda")
        full = torch.zeros(slots * sgl._row_bytes(p), dtype=torch.uint8, device="cuda")
        short = full[:-1]
        q, o, lse = new.clone(), torch.empty_like(new), torch.empty(B, hkv, device="cuda")
        for k, v in ((short, full), (full, short)):
            with pytest.raises(ValueError):
                sgl.sgl_kv_append(None, p, None, new, new, k, v, table, lens, None, None, ws)
            with pytest.raises(ValueError):
                sgl.sgl_extend_attn_kvwrite(q, new, new, k, v, table, zero, lens, p, o, lse, ws)
        assert not full.any()
        sgl.sgl_kv_append(None, p, None, new, new, full, full.clone(), table, lens, None, None, ws)
        sgl.sgl_check(ws)
        assert full.any()
    p = sgl.make_params(sgl.SGL_DTYPE_BF16, B, hkv, hkv, d, slots)
    small = torch.zeros(slots, row, dtype=torch.uint8, device="cuda")       # a 4-bit pool in a bf16 call
    new = torch.ones(B, hkv, d, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        sgl.sgl_kv_append(None, p, None, new, new, small, small, table, lens, None, None, ws)
    m = sgl.make_mla_params(B, 16, slots)
    kv = torch.ones(B, 576, dtype=torch.bfloat16, device="cuda")
    pool = torch.zeros(slots, 576, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        sgl.sgl_mla_kv_append(None, m, None, kv, pool[:-1], table, lens, None, None, ws)
    assert not pool.any() and not small.any()
    sgl.sgl_mla_kv_append(None, m, None, kv, pool, table, lens, None, None, ws)
    sgl.sgl_check(ws)
    assert np.array_equal(pool.any(1).nonzero()[:, 0].cpu().numpy(), [0, 4])
