"""Pools without rows: what would read an E4M3 row is refused on the host."""

import numpy as np
import pytest

import radixattention_prefix_shared_radix_gb300 as sgl


def _plan(dtype, slots, shared):
    table = np.zeros((20, 300), dtype=np.int32)
    table[:] = np.arange(300)
    if not shared:
        table += 300 * np.arange(20, dtype=np.int32)[:, None]
    lens = np.full(20, 300, dtype=np.int32)
    g = sgl.sgl_groups_create()
    try:
        sgl.sgl_groups_from_table(table, lens, g)
        return sgl.sgl_decode_plan(sgl.make_params(dtype, 20, 32, 8, 128, slots), lens, sgl.sgl_groups_view(g))
    finally:
        sgl.sgl_groups_destroy(g)


def test_tiles():
    with pytest.raises(sgl.SglError) as e:
        _plan(sgl.SGL_DTYPE_BF16_FP8KV, 0, True)
    assert e.value.status == -1
    assert sgl.sgl_plan_info(_plan(sgl.SGL_DTYPE_BF16_FP8KV, 1, True))["num_wide_items"] > 0
    # streams and 4-bit tiles read nothing for a slot outside the pool
    assert sgl.sgl_plan_info(_plan(sgl.SGL_DTYPE_BF16_FP8KV, 0, False))["num_wide_items"] == 0
    assert sgl.sgl_plan_info(_plan(sgl.SGL_DTYPE_BF16_FP4KV, 0, True))["num_wide_items"] > 0


def test_extend():
    import ctypes
    p = sgl.make_params(sgl.SGL_DTYPE_BF16_FP8KV, 1, 32, 8, 128, 0, host_prefix_lens=[0], host_extend_lens=[4])
    # (addresses that nothing may touch)
    assert sgl._lib().sgl_extend_attn(0x1000, 0x2000, 0x3000, 0x4000, 64, 0x5000, 0x5000, ctypes.byref(p), 0x6000, 0x7000,
                                      0x8000, 256, None) == -1
