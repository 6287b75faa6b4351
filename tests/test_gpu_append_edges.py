"""4-bit rows of values at the ends of bf16's range, byte for byte the format's definition (``oracle.fp4``)."""

import numpy as np
import pytest
import torch

import radixattention_prefix_shared_radix_gb300 as sgl
from oracle import fp4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from radixattention_prefix_shared_radix_gb300 import build
    build.build()


TOP = float(torch.finfo(torch.bfloat16).max)


@pytest.mark.parametrize("scale", [1.0, 0.16, 0.01, 1e-3, 1e-18, 2e-19, 1e-30, 1e-38, 1e-42, 1e18, 3e19, 1e37])
@pytest.mark.parametrize("write", [False, True])
def test_large_finite_values_into_4_bits(scale, write):
    """A block's scale is NaN only where a value is NaN: finite values saturate, whatever the tensor's scale, and keep
    their signs; small ones go to zero."""
    hkv, d = 2, 64
    tops = [TOP, 3e38, 1e38, 2.43e38, 2.7e37, 2.0 ** 60, 2.0 ** 59, 1.0, 2.0 ** -60, 1e-30, 1e-37, 1e-40]
    x = torch.zeros(len(tops), hkv, d)
    for r, t in enumerate(tops):
        x[r, 0, :16] = t * torch.linspace(-1, 1, 16)
        x[r, 0, 16:32] = torch.tensor([t, -t] * 8)
        x[r, 0, 32:48] = torch.tensor([t, -1.0, 1e-3, 0.0] * 4)
        x[r, 0, 48:] = torch.tensor([-t] + [0.0] * 15)
        x[r, 1] = x[r, 0].flip(0) * 0.37
    x = x.bfloat16()
    assert x.isfinite().all()
    n = len(tops)
    params = sgl.make_params(sgl.SGL_DTYPE_BF16_FP4KV, 1, 2, hkv, d, n, k_scale=scale, v_scale=scale,
                             host_prefix_lens=[0], host_extend_lens=[n])
    kp, vp = (torch.full((n, fp4.row_bytes(hkv, d)), 0xFF, dtype=torch.uint8, device="cuda") for _ in "kv")
    table = torch.arange(n, dtype=torch.int32, device="cuda")[None].contiguous()
    zero, ext = (torch.tensor([i], dtype=torch.int32, device="cuda") for i in (0, n))
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    if write:
        q = torch.zeros(n, 2, d, dtype=torch.bfloat16, device="cuda")
        sgl.sgl_extend_attn_kvwrite(q, x.cuda(), (-x).cuda(), kp, vp, table, zero, ext, params, torch.empty_like(q),
                                    torch.zeros(n, 2, device="cuda"), ws)
    else:
        sgl.sgl_kv_append(None, params, None, x.cuda(), (-x).cuda(), kp, vp, table, zero, ext, None, ws)
    sgl.sgl_check(ws)
    used = hkv * (d // 2 + d // 16)
    for pool, y in ((kp, x), (vp, -x)):
        got, want = fp4.unpack(pool.cpu().numpy(), hkv, d), fp4.quantise(y.float().numpy(), scale)
        assert np.array_equal(got[1], want[1])
        assert np.array_equal(got[0], want[0])
        assert (pool.cpu().numpy()[:, used:] == 0xFF).all()
