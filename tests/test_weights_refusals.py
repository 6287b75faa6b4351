"""Refusals of the weights and of the eviction: raw calls with addresses that nothing may touch, refused on the host."""

import ctypes

import numpy as np
import pytest

import radixattention_prefix_shared_radix_gb300 as sgl
from oracle import evict as oevict
from radixattention_prefix_shared_radix_gb300 import build as sglbuild


@pytest.fixture(scope="module", autouse=True)
def _built():
    sglbuild.build()


A, B, C, D, W = (0x10000 * i for i in range(1, 6))


def test_weights_refuse_before_any_gpu_work():
    lib = sgl._lib()
    p = sgl.make_params(sgl.SGL_DTYPE_BF16, 4, 8, 2, 128, 1000)
    ok = dict(q=A, lse=B, kp=C, t=D, ld=64, lens=A, ext=None, p=p, window=0, si=B, so=C, sld=64, decay=1.0, ws=W, wsb=256)

    def weights(**kw):
        a = dict(ok, **kw)
        a["p"] = ctypes.byref(a["p"]) if a["p"] else None
        return lib.sgl_attn_weights(*[a[x] for x in ("q", "lse", "kp", "t", "ld", "lens", "ext", "p", "window", "si", "so",
                                                     "sld", "decay", "ws", "wsb")], None)
    assert weights(p=None) == -1 and weights(ld=-1) == -1 and weights(sld=-1) == -1 and weights(window=-1) == -1
    for x in (-0.5, float("nan"), float("inf")):
        assert weights(decay=x) == -1
    assert weights(ws=None) == -7 and weights(ws=W + 16) == -7 and weights(wsb=128) == -7
    assert weights(lens=None) == -1 and weights(q=None) == -1 and weights(lse=None) == -1 and weights(kp=None) == -1
    assert weights(t=None) == -1 and weights(so=None) == -1 and weights(q=A + 8) == -1 and weights(kp=C + 8) == -1
    assert weights(ext=A) == -1                    # no host copies of the lengths
    assert weights(ld=0) == 0 and weights(sld=0) == 0
    assert weights(p=sgl.make_params(7, 4, 8, 2, 128, 1000)) == -3
    assert weights(p=sgl.make_params(sgl.SGL_DTYPE_BF16, 4, 8, 2, 96, 1000)) == -3
    assert weights(p=sgl.make_params(sgl.SGL_DTYPE_BF16, 4, 6, 2, 128, 1000)) == -3
    assert weights(p=sgl.make_params(sgl.SGL_DTYPE_BF16_FP8KV, 4, 8, 2, 128, 1000, k_scale=0.0)) == -1
    assert weights(p=sgl.make_params(sgl.SGL_DTYPE_BF16, 0, 8, 2, 128, 1000), lens=None) == 0

    def chunk(pre, ext, **kw):
        q = sgl.make_params(sgl.SGL_DTYPE_BF16, 2, 8, 2, 128, 1000, host_prefix_lens=pre, host_extend_lens=ext)
        return weights(p=q, ext=A, **dict(dict(wsb=1 << 30), **kw))
    assert chunk([60, 3], [5, 1]) == -1            # past the table
    assert chunk([-1, 3], [5, 1]) == -1 and chunk([1, 3], [5, -1]) == -1
    assert chunk([10, 3], [5, 1], sld=14) == -1
    assert chunk([0, 0], [0, 0]) == 0              # nothing cached, nothing new
    assert chunk([10, 3], [5, 1], q=None) == -1 and chunk([10, 3], [5, 1], wsb=128) == -7


def test_workspace_sizes():
    p = sgl.make_params(sgl.SGL_DTYPE_BF16, 2, 8, 2, 128, 1000)
    assert sgl.sgl_attn_weights_workspace_bytes(p) == 256
    q = sgl.make_params(sgl.SGL_DTYPE_BF16, 2, 8, 2, 128, 1000, host_prefix_lens=[100, 0], host_extend_lens=[300, 7])
    n = sgl.sgl_attn_weights_workspace_bytes(q)
    assert n >= 256 and n % 256 == 0
    lib = sgl._lib()
    size = ctypes.c_size_t()
    assert lib.sgl_attn_weights_workspace_bytes(ctypes.byref(p), -1, ctypes.byref(size)) == -1
    assert lib.sgl_attn_weights_workspace_bytes(ctypes.byref(p), 0, None) == -1
    bad = sgl.make_params(sgl.SGL_DTYPE_BF16, 2, 8, 2, 128, 1000, host_prefix_lens=[100, 0], host_extend_lens=[300, -7])
    assert lib.sgl_attn_weights_workspace_bytes(ctypes.byref(bad), 0, ctypes.byref(size)) == -1
    bad = sgl.make_params(sgl.SGL_DTYPE_BF16, 2, 8, 2, 128, 1000, host_extend_lens=[300, 7])
    assert lib.sgl_attn_weights_workspace_bytes(ctypes.byref(bad), 0, ctypes.byref(size)) == -1


def test_eviction_refuses_before_any_gpu_work():
    lib = sgl._lib()
    ok = dict(p=sgl.SglEvictParams(4, 1, 0, 0), s=A, sld=64, t=B, ld=64, pos=None, lens=C, bud=D, so=A, to=B, po=None, lo=C,
              ev=None, eld=0, cnt=None, ws=W, wsb=256)

    def evict(**kw):
        a = dict(ok, **kw)
        a["p"] = ctypes.byref(a["p"]) if a["p"] else None
        return lib.sgl_kv_evict(*[a[x] for x in ("p", "s", "sld", "t", "ld", "pos", "lens", "bud", "so", "to", "po", "lo",
                                                 "ev", "eld", "cnt", "ws", "wsb")], None)
    for bad in ((-1, 1, 0, 0), (4, 0, 0, 0), (4, 1, -1, 0), (4, 1, 0, -1)):
        assert evict(p=sgl.SglEvictParams(*bad)) == -1
    assert evict(p=None) == -1 and evict(sld=-1) == -1 and evict(ld=-1) == -1 and evict(eld=-1) == -1
    assert evict(ws=None) == -7 and evict(ws=W + 16) == -7 and evict(wsb=128) == -7
    for x in ("s", "t", "lens", "bud", "so", "to", "lo"):
        assert evict(**{x: None}) == -1
    assert evict(pos=A) == -1 and evict(po=A) == -1
    assert evict(ld=1 << 20, sld=1 << 20) == -3 and evict(ld=1 << 31, sld=1 << 31) == -3
    assert evict(p=sgl.SglEvictParams(0, 1, 0, 0), lens=None) == 0


def test_the_oracles_selection():
    """By hand: pages, sinks, recent tokens, ties, NaN."""
    s = np.array([5, 1, 1, 9, 1, 2, 7], dtype=np.float32)
    assert oevict.keep(s, 7).all() and oevict.keep(s, 8).all()
    assert np.nonzero(oevict.keep(s, 3))[0].tolist() == [0, 3, 6]
    assert np.nonzero(oevict.keep(s, 5))[0].tolist() == [0, 1, 3, 5, 6]          # (the earliest of the ones)
    assert np.nonzero(oevict.keep(s, 4, sinks=2, recent=1))[0].tolist() == [0, 1, 3, 6]
    assert np.nonzero(oevict.keep(s, 0, sinks=1, recent=2))[0].tolist() == [0, 5, 6]
    assert np.nonzero(oevict.keep(s, 4, page=2))[0].tolist() == [2, 3, 6]        # (the last page is not full)
    assert np.nonzero(oevict.keep(s, 5, page=2))[0].tolist() == [0, 1, 2, 3, 6]
    s[3] = np.nan
    assert np.nonzero(oevict.keep(s, 2))[0].tolist() == [0, 6]


def test_the_oracles_weights():
    """One row that sees everything: its weights are the softmax, and sum to one."""
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((3, 4, 8)), rng.standard_normal((10, 2, 8))
    lse = np.zeros((3, 4))
    for i in range(3):
        for h in range(4):
            lse[i, h] = np.log(np.exp(0.3 * k[:8 + i, h // 2] @ q[i, h]).sum())
    w, tol = oevict.weights(q, lse, k, 7, 0.3)
    assert abs(w.sum() - 12) < 1e-12 and (tol > 0).all()
    assert abs(w[9] - sum(np.exp(0.3 * k[9, h // 2] @ q[2, h] - lse[2, h]) for h in range(4))) < 1e-12
