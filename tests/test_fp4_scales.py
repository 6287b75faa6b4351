"""Tensor scales of 4-bit pools: what the quantiser divides by is six of them, which must be a finite number."""

import numpy as np
import pytest

import radixattention_prefix_shared_radix_gb300 as sgl

LARGEST = float(np.nextafter(np.float32(2.0 ** 128 / 6), np.float32(0)))     # six of it round to a finite number


@pytest.mark.parametrize("which", ["k_scale", "v_scale"])
@pytest.mark.parametrize("scale,ok", [(1.0, True), (1e-45, True), (LARGEST, True), (6e37, False), (1e38, False),
                                      (3.4e38, False), (float("inf"), False), (float("nan"), False), (0.0, False),
                                      (-1.0, False)])
def test_scales(which, scale, ok):
    p = sgl.make_params(sgl.SGL_DTYPE_BF16_FP4KV, 1, 8, 2, 128, 100, **{which: scale})
    if ok:
        assert np.isfinite(np.float32(6) * np.float32(scale))
        assert sgl.sgl_extend_workspace_bytes(p) > 0
        return
    with pytest.raises(sgl.SglError) as e:
        sgl.sgl_extend_workspace_bytes(p)
    assert e.value.status == -1
    with pytest.raises(sgl.SglError) as e:
        sgl.sgl_decode_plan(p, np.array([4], dtype=np.int32), sgl.SglPrefixGroups())
    assert e.value.status == -1
