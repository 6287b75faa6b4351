"""Arguments of the append that are refused before anything is looked at on a device."""

import pytest

import radixattention_prefix_shared_radix_gb300 as sgl


def test_positions_need_a_rotation():
    p = sgl.make_params(sgl.SGL_DTYPE_BF16, 4, 2, 2, 64, 16)
    with pytest.raises(TypeError, match="positions need a rope"):
        sgl.sgl_kv_append(None, p, *[None] * 10, positions=[0, 1, 2, 3])
