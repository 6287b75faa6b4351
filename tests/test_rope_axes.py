"""Rotary positions with several axes, and the append at given positions.

Rotated rows are held to the float64 oracle within the bound that tests/test_rope.py derives, one axis after the other
(the pairs of other axes masked); appended ones to the bytes of the rows that `sgl_rope` gives.
"""

import ctypes

import numpy as np
import pytest
import torch

import radixattention_prefix_shared_radix_gb300 as sgl
from oracle import rope as orope
from radixattention_prefix_shared_radix_gb300 import build as sglbuild
from tests.test_rope import KINDS, SCALINGS, _bytes, _pool, _rope, _stored

gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    sglbuild.build()


def _axes(d, rot, axes, off=0, pairs=False, scaling="none", arrange="blocks", own=False, theta=10000.0):
    """(library handle, frequency and axis of each pair, amplitude)"""
    kind, kw = SCALINGS[scaling]
    r = sgl.sgl_rope_create(d, rot, off, sgl.SGL_ROPE_PAIRS if pairs else sgl.SGL_ROPE_HALF, kind, theta,
                            kw.get("factor", 1.0), kw.get("original", 0), kw.get("low", 0.0), kw.get("high", 0.0), 0.0,
                            axes, sgl.SGL_ROPE_AXES_TURNS if arrange == "turns" else sgl.SGL_ROPE_AXES_BLOCKS, own)
    if arrange == "blocks":
        axis = np.repeat(np.arange(len(axes)), axes)
    else:
        axis = np.array([a for i in range(max(axes)) for a in range(len(axes)) if i < axes[a]])
    freq = orope.frequencies(rot, theta, scaling, **kw)
    if own:
        for a, n in enumerate(axes):
            freq[axis == a] = orope.frequencies(2 * n, theta, scaling, **kw)
    return r, freq, axis, (0.1 * np.log(kw["factor"]) + 1.0 if scaling == "yarn" else 1.0)


def _check(out, x, pos, rot, off, pairs, freq, axis, amp):
    """pos [axes, n] (numpy); rows at a negative position are passed over."""
    live = (pos >= 0).all(0)
    xd = x.double().cpu().numpy()[live]
    h = rot // 2
    ia = np.arange(off, off + rot, 2) if pairs else np.arange(off, off + h)
    ib = ia + (1 if pairs else h)
    t = pos[axis][:, live].T[:, None, :].astype(np.float64) * freq
    c, s = amp * np.cos(t), amp * np.sin(t)
    a, b = xd[..., ia], xd[..., ib]
    ref, size, far = xd.copy(), np.zeros_like(xd), np.zeros_like(xd)
    ref[..., ia], ref[..., ib] = a * c - b * s, b * c + a * s
    size[..., ia] = size[..., ib] = np.abs(a) + np.abs(b)
    far[..., ia] = far[..., ib] = pos.max(initial=0) * 2.0 ** -51
    half = 2.0 ** -8 if out.dtype == torch.bfloat16 else 2.0 ** -24
    tol = size * amp * (2.0 ** -22 + far) * (1 + half) + np.abs(ref) * half + 1e-30
    err = np.abs(out.double().cpu().numpy()[live] - ref)
    assert (err <= tol).all(), "worst %.3g of the bound" % (err / tol).max()


# ------------------------------------------------------------------ refusals (CPU)
@pytest.mark.parametrize("kw,status", [
    (dict(axes=(16, 16), rot_dim=32), -1), (dict(axes=(0, 32)), -1), (dict(axes=(-1, 33)), -1),
    (dict(axes=(16, 16), arrange=2), -3), (dict(axes=(31, 1), own_ladder=True, scaling=2, factor=2.0), -1),
    (dict(axes=(16, 16), head_dim=0), -1), (dict(axes=(16, 16), scaling=9), -3), (dict(axes=(20, 11)), -1),
    (dict(axes=(33,)), -1), (dict(axes=(2 ** 30, 2 ** 30, 2 ** 30, 2 ** 30)), -1)])
def test_create_refuses(kw, status):
    with pytest.raises(sgl.SglError) as e:
        sgl.sgl_rope_create(**{"head_dim": 64, "rot_dim": 64, **kw})
    assert e.value.status == status


def test_create_takes_one_to_four_axes():
    for axes in ((), (8, 8, 8, 4, 4)):
        with pytest.raises(ValueError):
            sgl.sgl_rope_create(64, axes=axes)
    lib = sgl._lib()
    p = sgl.SglRopeParams(64, 64, 0, 0, 0, 10000.0, 1.0, 0, 0.0, 0.0, 0.0)
    h = ctypes.c_void_p()
    for n, sections in ((0, (32, 0, 0, 0)), (5, (8, 8, 8, 8)), (-1, (32, 0, 0, 0))):
        a = sgl.SglRopeAxes(n, (ctypes.c_int32 * 4)(*sections), 0, 0)
        assert lib.sgl_rope_create_axes(ctypes.byref(p), ctypes.byref(a), ctypes.byref(h)) == -1
    a = sgl.SglRopeAxes(1, (ctypes.c_int32 * 4)(32, 0, 0, 0), 0, 2)
    assert lib.sgl_rope_create_axes(ctypes.byref(p), ctypes.byref(a), ctypes.byref(h)) == -1
    assert lib.sgl_rope_create_axes(None, ctypes.byref(a), ctypes.byref(h)) == -1
    assert lib.sgl_rope_create_axes(ctypes.byref(p), None, ctypes.byref(h)) == -1
    for axes in ((32,), (16, 16), (10, 11, 11), (1, 1, 1, 29)):
        assert sgl.sgl_rope_create(64, axes=axes).axes == len(axes)


def test_append_at_refuses_before_any_gpu_work():
    lib = sgl._lib()
    r = sgl.sgl_rope_create(128, axes=(16, 24, 24))
    p = sgl.make_params(sgl.SGL_DTYPE_BF16, 4, 8, 2, 128, 1000)
    A, B, C, D, W = (0x10000 * i for i in range(1, 6))
    ok = dict(rope=r.handle, p=p, q=A, qs=1024, k=B, ks=256, v=C, vs=256, kp=D, vp=D, t=A, ld=64, lens=A, ext=None, pos=A,
              n=4, qo=A, qos=1024, ws=W, wsb=256)

    def append(**kw):
        a = dict(ok, **kw)
        a["p"] = ctypes.byref(a["p"])
        return lib.sgl_kv_append_at(*[a[x] for x in ("rope", "p", "q", "qs", "k", "ks", "v", "vs", "kp", "vp", "t", "ld",
                                                     "lens", "ext", "pos", "n", "qo", "qos", "ws", "wsb")], None)
    assert append(rope=None) == -1 and append(pos=None) == -1 and append(n=5) == -1 and append(k=None) == -1
    assert append(ws=W + 16) == -7 and append(ks=252) == -1 and append(qo=None) == -1
    assert append(n=0) == 0 and append(n=0, pos=None) == 0
    other = sgl.sgl_rope_create(64, axes=(16, 16))
    assert append(rope=other.handle) == -1


# ------------------------------------------------------------------ rotation (GPU)
@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,rot,off,pairs,scaling,axes", [
    (128, 128, 0, False, "none", (16, 24, 24)), (128, 128, 0, True, "banded", (24, 20, 20)),
    (64, 64, 0, False, "none", (16, 16)), (64, 32, 32, False, "yarn", (1, 14, 1)), (128, 96, 32, True, "linear", (5, 40, 2, 1)),
    (256, 256, 0, False, "ntk", (64, 30, 34)), (80, 64, 16, False, "none", (32,)), (576, 64, 512, True, "none", (2, 15, 15)),
    (16, 16, 0, False, "none", (2, 2, 2, 2)), (1024, 256, 512, False, "none", (40, 44, 44))])
@pytest.mark.parametrize("arrange", ["blocks", "turns"])
@pytest.mark.parametrize("own", [False, True])
def test_rotation(dtype, d, rot, off, pairs, scaling, axes, arrange, own):
    if own and scaling == "ntk":
        axes = tuple(max(a, 2) for a in axes)
    r, freq, axis, amp = _axes(d, rot, axes, off, pairs, scaling, arrange, own)
    g = torch.Generator().manual_seed(d + rot)
    for n, hq, hk in ((1, 3, 1), (37, 5, 2), (310, 4, 1)):
        x = torch.randn(n, (hq + 2 * hk) * d, generator=g).to(dtype).cuda()
        q, k = x[:, :hq * d].unflatten(1, (hq, d)), x[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
        pos = torch.randint(0, 1 << 20, (len(axes), n), generator=g, dtype=torch.int32)
        pos[:, 0] = 0
        if n > 2:
            pos[len(axes) - 1, 1], pos[0, 2] = -1, -7
            pos[0, 3] = 2 ** 31 - 1
        qo = torch.full((n, hq, d), 7.0, dtype=dtype, device="cuda")
        ko = torch.full((n, hk, d), 7.0, dtype=dtype, device="cuda")
        sgl.sgl_rope(r, q, k, pos.cuda(), qo, ko)
        p = pos.numpy().astype(np.int64)
        _check(qo, q, p, rot, off, pairs, freq, axis, amp)
        _check(ko, k, p, rot, off, pairs, freq, axis, amp)
        if n > 2:
            assert (qo[1:3] == 7).all() and (ko[1:3] == 7).all()     # negative on any axis: left alone
        y = x.clone()
        sgl.sgl_rope(r, y[:, :hq * d].unflatten(1, (hq, d)), y[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d)), pos.cuda())
        live = (pos >= 0).all(0).cuda()[:, None]
        assert torch.equal(y[:, :hq * d], torch.where(live, qo.flatten(1), x[:, :hq * d]))
        assert torch.equal(y[:, hq * d:(hq + hk) * d], torch.where(live, ko.flatten(1), x[:, hq * d:(hq + hk) * d]))
        assert torch.equal(y[:, (hq + hk) * d:], x[:, (hq + hk) * d:])


@gpu
@pytest.mark.parametrize("arrange", ["blocks", "turns"])
def test_equal_positions_on_every_axis_are_a_rotation_with_one(arrange):
    """Text stands at one position on all axes: with the shared ladder the same bits as without axes."""
    g = torch.Generator().manual_seed(2)
    q = torch.randn(300, 9, 128, generator=g).bfloat16().cuda()
    pos = torch.randint(0, 1 << 17, (300,), generator=g, dtype=torch.int32).cuda()
    one, _, _ = _rope(128, 128, scaling="banded")
    r, *_ = _axes(128, 128, (16, 24, 24), scaling="banded", arrange=arrange)
    single, *_ = _axes(128, 128, (64,), scaling="banded", arrange=arrange)
    a, b, c, e = (torch.empty_like(q) for _ in range(4))
    sgl.sgl_rope(one, q, None, pos, a)
    sgl.sgl_rope(r, q, None, pos.repeat(3, 1), b)
    sgl.sgl_rope(single, q, None, pos, c)
    sgl.sgl_rope(single, q, None, pos[None], e)
    assert torch.equal(a, b) and torch.equal(a, c) and torch.equal(a, e)


# ------------------------------------------------------------------ append (GPU)
@gpu
@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("hq,hkv,d,rot,off,pairs,axes", [(8, 8, 128, 128, 0, False, (16, 24, 24)),
                                                         (10, 5, 64, 32, 32, False, (8, 8)), (8, 1, 64, 64, 0, True, (32,)),
                                                         (16, 2, 128, 64, 0, True, (2, 10, 10, 10))])
@pytest.mark.parametrize("decode", [False, True])
def test_append_at(kind, hq, hkv, d, rot, off, pairs, axes, decode):
    rng = np.random.default_rng(hq * d + rot)
    B = 9
    ext = np.ones(B, dtype=np.int64) if decode else np.array([3, 0, 1, 40, 0, 17, 64, 1, 0])
    pre = rng.integers(0, 300, B)
    rows = int(ext.sum())
    n = rows if decode else rows + 13              # a batch padded to its bucket
    ld, slots = 400, 700
    order = rng.permutation(slots)
    table = np.full((B, ld), -1, dtype=np.int32)
    who = [(r, i) for r in range(B) for i in range(ext[r])]
    for at, (r, i) in enumerate(who):
        table[r, pre[r] + i] = order[at]
    dt = torch.float32 if kind == "f32" else torch.bfloat16
    g = torch.Generator().manual_seed(rot)
    qkv = torch.randn(n, (hq + 2 * hkv) * d, generator=g).to(dt).cuda()
    q, k, v = (t.unflatten(1, (-1, d)) for t in qkv.split((hq * d, hkv * d, hkv * d), 1))
    r, freq, axis, amp = _axes(d, rot, axes, off, pairs, "banded", "turns" if decode else "blocks", own=decode)
    pos = torch.randint(0, 1 << 18, (len(axes), n), generator=g, dtype=torch.int32)
    pos[len(axes) - 1, rows // 2] = -1             # a row that is left out
    live = np.array([i for i in range(rows) if i != rows // 2])
    ks, vs = 0.37, 1.3
    params = sgl.make_params(KINDS[kind], B, hq, hkv, d, slots, k_scale=ks, v_scale=vs)
    kp, vp = _pool(kind, slots, hkv, d, 1), _pool(kind, slots, hkv, d, 2)
    kb, vb = _bytes(kp), _bytes(vp)
    qo = torch.full((n, hq, d), 7.0, dtype=dt, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    lens = torch.from_numpy((pre + 1 if decode else pre).astype(np.int32)).cuda()
    extd = None if decode else torch.from_numpy(ext.astype(np.int32)).cuda()
    td = torch.from_numpy(table).cuda()
    sgl.sgl_kv_append_at(r, params, q, k, v, kp, vp, td, lens, extd, pos.cuda(), qo, ws)
    sgl.sgl_check(ws)
    _check(qo[:rows], q[:rows], pos.numpy()[:, :rows].astype(np.int64), rot, off, pairs, freq, axis, amp)
    assert (qo[rows:] == 7).all() and (qo[rows // 2] == 7).all()
    kr, qr = torch.full((n, hkv, d), 7.0, dtype=dt, device="cuda"), torch.full_like(qo, 7.0)
    sgl.sgl_rope(r, q, k, pos.cuda(), qr, kr)
    assert torch.equal(qr[:rows], qo[:rows])
    to = order[live]
    kb[to] = _stored(kind, kr[live], ks, hkv, d, kb[to])
    vb[to] = _stored(kind, v[live], vs, hkv, d, vb[to])
    assert np.array_equal(_bytes(kp), kb) and np.array_equal(_bytes(vp), vb)
    # at the places in the rows, on every axis: the append without positions
    place = np.concatenate([[pre[a] + i for a, i in who], np.zeros(n - rows)]).astype(np.int32)
    k1, v1, k2, v2 = (_pool(kind, slots, hkv, d, i) for i in (1, 2, 1, 2))
    q1, q2 = torch.zeros_like(qo), torch.zeros_like(qo)
    sgl.sgl_kv_append_at(r, params, q, k, v, k1, v1, td, lens, extd,
                         torch.from_numpy(place).cuda().repeat(len(axes), 1), q1, ws)
    sgl.sgl_kv_append(r, params, q, k, v, k2, v2, td, lens, extd, q2, ws)
    sgl.sgl_check(ws)
    assert torch.equal(q1, q2) and np.array_equal(_bytes(k1), _bytes(k2)) and np.array_equal(_bytes(v1), _bytes(v2))


@gpu
def test_append_at_in_a_graph_follows_lengths_and_positions():
    B, hkv, d, slots, ld = 3, 2, 128, 64, 16
    r, freq, axis, amp = _axes(d, d, (16, 24, 24))
    params = sgl.make_params(sgl.SGL_DTYPE_BF16, B, 2, hkv, d, slots)
    table = torch.randperm(slots)[:B * ld].view(B, ld).to(torch.int32).cuda()
    k, v = (torch.randn(B, hkv, d, device="cuda").bfloat16() for _ in "kv")
    kp, vp = (torch.zeros(slots, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    lens = torch.tensor([1, 5, 9], dtype=torch.int32, device="cuda")
    pos = torch.randint(0, 5000, (3, B), dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            sgl.sgl_kv_append_at(r, params, None, k, v, kp, vp, table, lens, None, pos, None, ws)
    del r
    for _ in range(3):
        kp.zero_()
        graph.replay()
        torch.cuda.synchronize()
        to = table.cpu().numpy()[np.arange(B), lens.cpu().numpy() - 1]
        _check(kp[to], k, pos.cpu().numpy().astype(np.int64), d, 0, False, freq, axis, amp)
        assert int(kp.flatten(1).any(1).sum()) == B
        lens += 1
        pos += 77
    sgl.sgl_check(ws)


@gpu
def test_python_arguments_are_checked():
    r = sgl.sgl_rope_create(64, axes=(10, 11, 11))
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(3, 4, dtype=torch.int32, device="cuda")
    sgl.sgl_rope(r, q, None, pos)
    p = sgl.make_params(sgl.SGL_DTYPE_BF16, 4, 2, 2, 64, 16)
    pool = torch.zeros(16, 2, 64, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(4, 8, dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    lens = torch.zeros(4, dtype=torch.int32, device="cuda")
    good = dict(rope=r, params=p, q=None, k_new=q, v_new=q, k_pool=pool, v_pool=pool, req_to_token=table, lens=lens,
                extend_lens=None, positions=pos, q_out=None, workspace=ws)
    for bad in (pos[:2], pos[0], pos[:, :3], pos.long(), pos.cpu(), torch.zeros(4, 3, dtype=torch.int32, device="cuda").T):
        with pytest.raises((TypeError, ValueError)):
            sgl.sgl_rope(r, q, None, bad)
        with pytest.raises((TypeError, ValueError)):
            sgl.sgl_kv_append_at(**dict(good, positions=bad))
    for bad in (dict(rope=None), dict(positions=None)):
        with pytest.raises(TypeError):
            sgl.sgl_kv_append_at(**dict(good, **bad))
    sgl.sgl_kv_append_at(**good)                  # (lengths of zero: nothing to append)
    sgl.sgl_check(ws)
    assert not pool.any()
