"""The workspace of the attention weights: what it grows with, and the lengths that are refused, by the call and by the
call that sizes its workspace alike."""

import ctypes

import pytest

import radixattention_prefix_shared_radix_gb300 as sgl
from radixattention_prefix_shared_radix_gb300 import build as sglbuild


@pytest.fixture(scope="module", autouse=True)
def _built():
    sglbuild.build()


def _params(pre, ext, hq=64, hkv=8, dtype=sgl.SGL_DTYPE_BF16, **kw):
    return sgl.make_params(dtype, len(ext), hq, hkv, 128, 1000, host_prefix_lens=pre, host_extend_lens=ext, **kw)


def _both(p, window=0):
    """(status of the sizing call, its bytes, status of a call without a pool: -1 where the lengths are taken)"""
    lib, size = sgl._lib(), ctypes.c_size_t(0)
    st = lib.sgl_attn_weights_workspace_bytes(ctypes.byref(p), window, ctypes.byref(size))
    A, ld = 0x10000, 1 << 33
    call = lib.sgl_attn_weights(A, A, None, A, ld, A, A, ctypes.byref(p), window, None, A, ld, 1.0, A, 256, None)
    return st, size.value, call


@pytest.mark.parametrize("pre,ext", [
    ([0], [32768]), ([0], [131072]), ([0], [524288]), ([0], [1 << 20]), ([0], [1 << 24]), ([1 << 20], [8192]),
    ([131072] * 8, [8192] * 8), ([0] * 16, [32768] * 16), ([0, 5, 300], [70, 0, 200000])])
@pytest.mark.parametrize("hq,hkv", [(64, 8), (32, 8), (8, 8), (8, 1)])
@pytest.mark.parametrize("dtype", [sgl.SGL_DTYPE_BF16, sgl.SGL_DTYPE_BF16_FP8KV, sgl.SGL_DTYPE_BF16_FP4KV])
def test_it_grows_with_positions_alone(pre, ext, hq, hkv, dtype):
    """2 KB for 256 positions of a request and KV head, and 160 MB (1 MiB an SM) besides, however many rows ask."""
    for window in (0, 4096):
        st, n, _ = _both(_params(pre, ext, hq, hkv, dtype), window)
        tiles = sum(-(-(a + b) // 256) for a, b in zip(pre, ext))
        assert st == 0 and 256 < n <= 256 + 2048 * hkv * tiles + 160_000_000


def test_small_calls_keep_an_item_for_each_sm():
    """8 x 512 after 4096, 64/8 heads: 18 tiles of 32 query blocks each, in runs of 16; the last two tiles hold new
    tokens, whose first block the second of them lets half of the runs pass."""
    n = sgl.sgl_attn_weights_workspace_bytes(_params([4096] * 8, [512] * 8))
    assert n == 256 + 2048 * 8 * 8 * (17 * 2 + 1)


@pytest.mark.parametrize("pre,ext,kw", [
    ([0], [(1 << 24) + 1], {}), ([0, 0], [1 << 23, (1 << 23) + 1], {}),                   # rows
    ([(1 << 26) - 1], [2], {}), ([1 << 26], [1], {}), ([2 ** 31 - 1], [2 ** 31 - 1], {}),     # a context
    ([1 << 26] * 8, [0] * 8, {"hkv": 8, "hq": 8}),                                            # all positions: 2^32 ..
])
def test_limits_are_those_of_the_call(pre, ext, kw):
    st, _, call = _both(_params(pre, ext, **kw))
    if sum(ext) or len(pre) < 8:
        assert st == -3 and call == -3
    else:                     # .. fit, with a workspace of no items
        assert st == 0 and call == -1
    more = _params(pre + [1], ext + [0], **kw)
    st, _, call = _both(more)
    assert st == -3 and call == -3


def test_limits_over_fp32_pools():
    f32 = sgl.SGL_DTYPE_F32
    assert _both(_params([0] * 65535, [1] * 65535, dtype=f32)) == (0, 256, -1)
    st, _, call = _both(_params([0] * 65536, [1] * 65536, dtype=f32))
    assert st == -3 and call == -3
    st, _, call = _both(_params([1 << 26], [1], dtype=f32))
    assert st == -3 and call == -3


def test_work_is_cut_for_the_sms_asked_for():
    """num_sms as in the attention calls' planning; 0 and 152 are one on the device that the kernels are for."""
    def items(pre, ext, n):          # of a KV head
        return (sgl.sgl_attn_weights_workspace_bytes(_params([pre], [ext], num_sms=n)) - 256) / 2048 / 8
    # 13 query blocks for each of two tiles: 208 of all heads, two an SM of 152, 13 an SM of 16
    assert [items(300, 200, n) for n in (0, 152, 16, 1)] == [14, 14, 2, 2]
    # 57 blocks for each of five tiles, four runs of 15 (152 SMs) or of 16; rows see the last three from block 13, 29
    # and 45 on: runs 0, 1 and 3 of 15, or 0, 1 and 2 of 16
    assert [items(300, 900, n) for n in (0, 152, 16, 1)] == [16, 16, 17, 17]
    long = {n: sgl.sgl_attn_weights_workspace_bytes(_params([0], [1 << 20], num_sms=n)) for n in (8, 152, 2 ** 31 - 1)}
    assert long[8] <= 256 + 2048 * 8 * 4096 + (8 << 20) and long[8] < long[152] < long[2 ** 31 - 1] < 1 << 33
