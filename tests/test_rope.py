"""Rotary positions and the append to the paged pools.

The rotation is held to the float64 oracle.  Its error, per output element of
a pair (a, b) with amplitude A: the fp32 angle (at most pi / 4) is off by
2^-25 of itself from the conversion, sine and cosine by one unit in the last
place (2^-24 at most below 1) and by 2^-24 from the amplitude; each product
and the sum round once (2^-24).  Together under 2^-22 (|a| + |b|) A, plus the
output's rounding, half a step: 2^-8 of the value for bf16, 2^-24 for fp32.

Appended rows are held to equality: the pools' bytes are those of the rotated
keys (which `sgl_rope` gives) and values, stored or quantised one by one.
"""

import ctypes

import numpy as np
import pytest
import torch

import radixattention_prefix_shared_radix_gb300 as sgl
from oracle import fp4, rope as orope
from oracle.fp8 import quantise_rows
from radixattention_prefix_shared_radix_gb300 import build as sglbuild

gpu = pytest.mark.gpu

SCALINGS = {
    "none": (sgl.SGL_ROPE_SCALE_NONE, {}),
    "linear": (sgl.SGL_ROPE_SCALE_LINEAR, dict(factor=4.0)),
    "ntk": (sgl.SGL_ROPE_SCALE_NTK, dict(factor=8.0)),
    "yarn": (sgl.SGL_ROPE_SCALE_YARN, dict(factor=16.0, original=4096, low=1.0, high=32.0)),
    "banded": (sgl.SGL_ROPE_SCALE_BANDED, dict(factor=8.0, original=8192, low=1.0, high=4.0)),
}


@pytest.fixture(scope="module", autouse=True)
def _built():
    sglbuild.build()


def _rope(d, rot, off=0, pairs=False, scaling="none", theta=10000.0, amplitude=0.0):
    """(library handle, frequencies, amplitude)"""
    kind, kw = SCALINGS[scaling]
    r = sgl.sgl_rope_create(d, rot, off, sgl.SGL_ROPE_PAIRS if pairs else sgl.SGL_ROPE_HALF, kind, theta,
                            kw.get("factor", 1.0), kw.get("original", 0), kw.get("low", 0.0), kw.get("high", 0.0),
                            amplitude)
    amp = amplitude or (0.1 * np.log(kw["factor"]) + 1.0 if scaling == "yarn" else 1.0)
    return r, orope.frequencies(rot, theta, scaling, **kw), amp


def _check_rotated(out, x, pos, rot, off, pairs, freq, amp):
    """`out` (torch) against the oracle's rotation of `x` (torch), within the bound above; rows at pos < 0 skipped."""
    live = pos >= 0
    xd = x.double().cpu().numpy()[live]
    ref = orope.rotate(xd, pos[live], freq, off, pairs, amp)
    h = rot // 2
    a = slice(off, off + rot, 2) if pairs else slice(off, off + h)
    b = slice(off + 1, off + rot, 2) if pairs else slice(off + h, off + rot)
    size = np.zeros_like(ref)
    size[..., a] = size[..., b] = np.abs(xd[..., a]) + np.abs(xd[..., b])
    half = 2.0 ** -8 if out.dtype == torch.bfloat16 else 2.0 ** -24
    # (angles: the library's frequency is the double nearest in turns, the
    # oracle's in radians; both are off by 2^-53 of the angle, at most 2^31 radians)
    far = np.abs(pos[live]).max(initial=0) * 2.0 ** -51
    tol = size * amp * (2.0 ** -22 + far) * (1 + half) + np.abs(ref) * half + 1e-30
    err = np.abs(out.double().cpu().numpy()[live] - ref)
    assert (err <= tol).all(), "worst %.3g of the bound" % (err / tol).max()


# ------------------------------------------------------------------ refusals (CPU)
def _status(fn, *args):
    with pytest.raises(sgl.SglError) as e:
        fn(*args)
    return e.value.status


@pytest.mark.parametrize("kw,status", [
    (dict(head_dim=0), -1), (dict(head_dim=64, rot_dim=80), -1), (dict(head_dim=64, rot_dim=64, rot_offset=16), -1),
    (dict(head_dim=64, rot_offset=-16, rot_dim=16), -1), (dict(head_dim=72, rot_dim=16), -3),
    (dict(head_dim=64, rot_dim=24), -3), (dict(head_dim=128, rot_dim=48), -3), (dict(head_dim=1024, rot_dim=512), -3),
    (dict(head_dim=2048, rot_dim=64), -3), (dict(head_dim=64, rot_dim=32, rot_offset=8), -3),
    (dict(head_dim=64, theta=1.0), -1), (dict(head_dim=64, theta=float("nan")), -1), (dict(head_dim=64, layout=2), -3),
    (dict(head_dim=64, scaling=5), -3), (dict(head_dim=64, scaling=1, factor=0.5), -1),
    (dict(head_dim=64, scaling=3, factor=4.0, low=1.0, high=32.0), -1),
    (dict(head_dim=64, scaling=4, factor=4.0, original_positions=4096, low=4.0, high=1.0), -1),
    (dict(head_dim=64, attention_factor=-1.0), -1), (dict(head_dim=64, attention_factor=1e39), -1),
])
def test_rope_create_refuses(kw, status):
    with pytest.raises(sgl.SglError) as e:
        sgl.sgl_rope_create(**kw)
    assert e.value.status == status


def test_calls_refuse_before_any_gpu_work():
    """Raw calls with addresses that nothing may touch: every one is refused on the host."""
    lib = sgl._lib()
    r = sgl.sgl_rope_create(128, 128)
    A, B, C, D = (0x10000 * i for i in range(1, 5))
    good = dict(rope=r.handle, dtype=1, q=A, qs=1024, hq=8, k=B, ks=256, hk=2, pos=C, n=4, qo=A, qos=1024, ko=B, kos=256)

    def rope(**kw):
        a = dict(good, **kw)
        return lib.sgl_rope(*[a[x] for x in ("rope", "dtype", "q", "qs", "hq", "k", "ks", "hk", "pos", "n", "qo", "qos",
                                              "ko", "kos")], None)
    assert rope(rope=None) == -1 and rope(n=-1) == -1 and rope(pos=None) == -1
    assert rope(dtype=2) == -3 and rope(dtype=3) == -3
    assert rope(q=None) == -1 and rope(q=A + 8, qo=A + 8) == -1 and rope(qs=1023, qos=1023) == -1
    assert rope(qs=1028, qos=1028) == -1           # rows off the 16-byte grid
    assert rope(qos=2048) == -1                    # in place with another stride
    assert rope(ko=None) == -1 and rope(hk=-1) == -1
    assert rope(n=0) == 0

    p = sgl.make_params(sgl.SGL_DTYPE_BF16_FP4KV, 4, 8, 2, 128, 1000, k_scale=1.0, v_scale=1.0)
    W = 0x50000
    ok = dict(rope=r.handle, p=p, q=A, qs=1024, k=B, ks=256, v=C, vs=256, kp=D, vp=D, t=A, ld=64, lens=A, ext=None, n=4,
              qo=A, qos=1024, ws=W, wsb=256)

    def append(**kw):
        a = dict(ok, **kw)
        a["p"] = ctypes.byref(a["p"])
        return lib.sgl_kv_append(*[a[x] for x in ("rope", "p", "q", "qs", "k", "ks", "v", "vs", "kp", "vp", "t", "ld",
                                                  "lens", "ext", "n", "qo", "qos", "ws", "wsb")], None)
    assert append(n=5) == -1                       # decode: at most one row per request
    assert append(n=-1) == -1 and append(k=None) == -1 and append(v=None) == -1 and append(t=None) == -1
    assert append(lens=None) == -1 and append(qo=None) == -1 and append(q=None) == -1
    assert append(ws=None) == -7 and append(ws=W + 16) == -7 and append(wsb=128) == -7
    assert append(kp=D + 4) == -1 and append(ks=252) == -1
    other = sgl.sgl_rope_create(64, 64)
    assert append(rope=other.handle) == -1         # another head width
    bad = sgl.make_params(sgl.SGL_DTYPE_BF16_FP4KV, 4, 8, 2, 128, 1000, k_scale=0.0, v_scale=1.0)
    assert append(p=bad) == -1
    assert append(p=sgl.make_params(7, 4, 8, 2, 128, 1000)) == -3
    assert append(n=0) == 0

    m = sgl.make_mla_params(4, 16, 1000)

    def mla(**kw):
        a = dict(dict(rope=None, p=m, q=A, qs=16 * 576, kv=B, kvs=576, kp=D, t=A, ld=64, lens=A, ext=None, n=4, qo=A,
                      qos=16 * 576, ws=W, wsb=256), **kw)
        a["p"] = ctypes.byref(a["p"])
        return lib.sgl_mla_kv_append(*[a[x] for x in ("rope", "p", "q", "qs", "kv", "kvs", "kp", "t", "ld", "lens",
                                                      "ext", "n", "qo", "qos", "ws", "wsb")], None)
    assert mla(rope=r.handle) == -1 and mla(kv=None) == -1 and mla(kp=None) == -1 and mla(n=5) == -1
    assert mla(p=sgl.make_mla_params(4, 8, 1000)) == -3 and mla(n=0) == 0

    assert _status(sgl.sgl_fp4_row_bytes, 8, 96) == -3 and _status(sgl.sgl_fp4_row_bytes, 0, 64) == -1
    assert [sgl.sgl_fp4_row_bytes(*a) for a in ((8, 128), (1, 64), (5, 64), (2, 128))] == \
        [fp4.row_bytes(*a) for a in ((8, 128), (1, 64), (5, 64), (2, 128))]


# ------------------------------------------------------------------ rotation (GPU)
@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,rot,off,pairs,scaling", [
    (128, 128, 0, False, "none"), (128, 128, 0, True, "banded"), (64, 32, 0, False, "yarn"), (64, 16, 32, False, "ntk"),
    (128, 96, 32, True, "linear"), (576, 64, 512, True, "none"), (576, 64, 512, False, "yarn"), (256, 256, 0, False, "none"),
    (80, 64, 16, False, "none"), (16, 16, 0, False, "none")])
def test_rotation(dtype, d, rot, off, pairs, scaling):
    r, freq, amp = _rope(d, rot, off, pairs, scaling)
    g = torch.Generator().manual_seed(d + rot)
    for n, hq, hk in ((1, 3, 1), (37, 5, 2), (3, 64, 8)):
        # columns of a fused projection
        x = torch.randn(n, (hq + 2 * hk) * d, generator=g).to(dtype).cuda()
        q, k = x[:, :hq * d].unflatten(1, (hq, d)), x[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
        pos = torch.randint(0, 1 << 20, (n,), generator=g, dtype=torch.int32)
        pos[0] = 0 if n == 1 else 2 ** 31 - 1
        if n > 2:
            pos[1], pos[2] = -1, 1
        pos = pos.cuda()
        qo = torch.full((n, hq, d), 7.0, dtype=dtype, device="cuda")
        ko = torch.full((n, hk, d), 7.0, dtype=dtype, device="cuda")
        sgl.sgl_rope(r, q, k, pos, qo, ko)
        p = pos.cpu().numpy().astype(np.int64)
        _check_rotated(qo, q, p, rot, off, pairs, freq, amp)
        _check_rotated(ko, k, p, rot, off, pairs, freq, amp)
        if n > 2:
            assert (qo[1] == 7).all() and (ko[1] == 7).all()     # a negative position: left alone
        # in place, in the fused matrix: the same bits, and nothing else changes
        y = x.clone()
        sgl.sgl_rope(r, y[:, :hq * d].unflatten(1, (hq, d)), y[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d)), pos)
        live = (pos >= 0)[:, None]
        assert torch.equal(y[:, :hq * d], torch.where(live, qo.flatten(1), x[:, :hq * d]))
        assert torch.equal(y[:, hq * d:(hq + hk) * d], torch.where(live, ko.flatten(1), x[:, hq * d:(hq + hk) * d]))
        assert torch.equal(y[:, (hq + hk) * d:], x[:, (hq + hk) * d:])
        # queries alone, keys alone
        q2, k2 = torch.full_like(qo, 7.0), torch.full_like(ko, 7.0)
        sgl.sgl_rope(r, q, None, pos, q2)
        sgl.sgl_rope(r, None, k, pos, None, k2)
        assert torch.equal(q2, qo) and torch.equal(k2, ko)


@gpu
@pytest.mark.parametrize("n", [2431, 2432, 2501])
def test_rotation_of_many_rows(n):
    """Both sides of the size from which a CTA takes four tokens."""
    r, freq, amp = _rope(64, 64)
    g = torch.Generator().manual_seed(n)
    q = torch.randn(n, 3, 64, generator=g).bfloat16().cuda()
    pos = torch.randint(0, 5000, (n,), generator=g, dtype=torch.int32).cuda()
    out = torch.empty_like(q)
    sgl.sgl_rope(r, q, None, pos, out)
    _check_rotated(out, q, pos.cpu().numpy().astype(np.int64), 64, 0, False, freq, amp)


@gpu
def test_python_arguments_are_checked():
    r = sgl.sgl_rope_create(64)
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in (lambda: sgl.sgl_rope(r, q.cpu(), None, pos), lambda: sgl.sgl_rope(r, q.half(), None, pos),
                lambda: sgl.sgl_rope(r, q, None, pos.long()), lambda: sgl.sgl_rope(r, q, None, pos[:3]),
                lambda: sgl.sgl_rope(r, q[..., :32], None, pos), lambda: sgl.sgl_rope(r, q.transpose(0, 1), None, pos),
                lambda: sgl.sgl_rope(r, q, q.float(), pos), lambda: sgl.sgl_rope(r, None, None, pos),
                lambda: sgl.sgl_rope(r, q, None, pos, k_out=q), lambda: sgl.sgl_rope(r, None, q, pos, q_out=q)):
        with pytest.raises((TypeError, ValueError)):
            bad()
    p = sgl.make_params(sgl.SGL_DTYPE_BF16, 4, 2, 2, 64, 16)
    pool = torch.zeros(16, 2, 64, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(4, 8, dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    good = dict(rope=r, params=p, q=None, k_new=q, v_new=q, k_pool=pool, v_pool=pool, req_to_token=table, lens=pos,
                extend_lens=None, q_out=None, workspace=ws)
    for bad in (dict(req_to_token=table[:3]), dict(req_to_token=table[0]), dict(req_to_token=table.long()),
                dict(lens=pos[:3]), dict(k_new=q[:3]), dict(v_new=q.float()), dict(k_pool=pool.cpu()),
                dict(extend_lens=pos.long()), dict(q=q[:, :1], q_out=q), dict(workspace=ws.cpu())):
        with pytest.raises((TypeError, ValueError)):
            sgl.sgl_kv_append(**dict(good, **bad))
    sgl.sgl_kv_append(**good)                     # (lengths of zero: nothing to append)
    sgl.sgl_check(ws)
    assert not pool.any()


# ------------------------------------------------------------------ append (GPU)
KINDS = {"f32": sgl.SGL_DTYPE_F32, "bf16": sgl.SGL_DTYPE_BF16, "fp8": sgl.SGL_DTYPE_BF16_FP8KV,
         "fp4": sgl.SGL_DTYPE_BF16_FP4KV}


def _pool(kind, slots, hkv, d, seed):
    g = torch.Generator().manual_seed(seed)
    if kind in ("fp4", "fp8"):
        shape = (slots, fp4.row_bytes(hkv, d)) if kind == "fp4" else (slots, hkv, d)
        return torch.randint(0, 256, shape, generator=g, dtype=torch.uint8).cuda()
    return torch.randn(slots, hkv, d, generator=g).to(torch.float32 if kind == "f32" else torch.bfloat16).cuda()


def _stored(kind, x, scale, hkv, d, before):
    """Bytes of the pool rows that hold `x` (torch [n, hkv, d]); a padded 4-bit row keeps its padding."""
    if kind in ("f32", "bf16"):
        return x.cpu().contiguous().view(torch.uint8).reshape(x.shape[0], -1).numpy()
    v = x.float().cpu().numpy()
    if kind == "fp8":
        return quantise_rows(v, scale).reshape(x.shape[0], -1)
    rows = fp4.pack(*fp4.quantise(v, scale))
    used = hkv * (d // 2 + d // 16)
    rows[:, used:] = before[:, used:]
    return rows


def _bytes(pool):
    return pool.contiguous().view(torch.uint8).reshape(pool.shape[0], -1).cpu().numpy()


@gpu
@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("hq,hkv,d,rot,off,pairs", [(8, 8, 128, 128, 0, False), (10, 5, 64, 32, 32, False),
                                                    (8, 1, 64, 16, 16, False), (12, 12, 128, 64, 16, False),
                                                    (8, 2, 128, 128, 0, True), (4, 4, 128, 0, 0, False)])
@pytest.mark.parametrize("decode", [False, True])
def test_append(kind, hq, hkv, d, rot, off, pairs, decode):
    rng = np.random.default_rng(hq * d + rot)
    B = 9
    ext = np.ones(B, dtype=np.int64) if decode else np.array([3, 0, 1, 40, 0, 17, 64, 1, 0])
    pre = rng.integers(0, 300, B)
    if decode:
        pre[4] = -1                                # a request without context
    rows = B if decode else int(ext.sum())
    n = rows if decode else rows + 13              # a batch padded to its bucket
    ld, slots = 400, 700
    order = rng.permutation(slots)
    table = np.full((B, ld), -1, dtype=np.int32)
    who = [(r, i) for r in range(B) for i in range(ext[r])]
    for at, (r, i) in enumerate(who):
        if pre[r] + i >= 0:
            table[r, pre[r] + i] = order[at]
    dt = torch.float32 if kind == "f32" else torch.bfloat16
    g = torch.Generator().manual_seed(rot)
    qkv = torch.randn(n, (hq + 2 * hkv) * d, generator=g)
    qkv[0, -16:] = 0                               # a block of zeros, one with an infinity, one with a NaN
    qkv[1, -16], qkv[2, -1] = float("inf"), float("nan")
    qkv = qkv.to(dt).cuda()
    q, k, v = (t.unflatten(1, (-1, d)) for t in qkv.split((hq * d, hkv * d, hkv * d), 1))
    r = freq = None
    amp = 1.0
    if rot:
        r, freq, amp = _rope(d, rot, off, pairs, "banded")
    ks, vs = 0.37, 1.3
    params = sgl.make_params(KINDS[kind], B, hq, hkv, d, slots, k_scale=ks, v_scale=vs)
    kp, vp = _pool(kind, slots, hkv, d, 1), _pool(kind, slots, hkv, d, 2)
    kb, vb = _bytes(kp), _bytes(vp)
    qo = torch.full((n, hq, d), 7.0, dtype=dt, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    lens = torch.from_numpy((pre + 1 if decode else pre).astype(np.int32)).cuda()
    extd = None if decode else torch.from_numpy(ext.astype(np.int32)).cuda()
    sgl.sgl_kv_append(r, params, q, k, v, kp, vp, torch.from_numpy(table).cuda(), lens, extd, qo, ws)
    sgl.sgl_check(ws)
    pos = np.array([pre[a] + i for a, i in who])
    live = np.nonzero(pos >= 0)[0]
    if rot:
        _check_rotated(qo[:rows], q[:rows], pos, rot, off, pairs, freq, amp)
        posd = torch.from_numpy(np.concatenate([pos, np.full(n - rows, -1)]).astype(np.int32)).cuda()
        kr, qr = torch.full((n, hkv, d), 7.0, dtype=dt, device="cuda"), torch.full_like(qo, 7.0)
        sgl.sgl_rope(r, q, k, posd, qr, kr)
        assert torch.equal(qr, qo)
    else:
        kr = k
        assert torch.equal(qo[live], q[live])
    assert (qo[rows:] == 7).all()                  # rows behind the last request
    to = np.array([table[who[i][0], pos[i]] for i in live])
    kb[to] = _stored(kind, kr[live], ks, hkv, d, kb[to])
    vb[to] = _stored(kind, v[live], vs, hkv, d, vb[to])
    got_k, got_v = _bytes(kp), _bytes(vp)
    if kind == "fp4":                              # codes of a block whose scale is NaN mean nothing
        for got, want in ((got_k, kb), (got_v, vb)):
            a, b = (fp4.unpack(x, hkv, d) for x in (got, want))
            assert np.array_equal(a[1], b[1])
            nan = np.repeat(b[1] & 0x7F == 0x7F, 16, -1)
            assert np.array_equal(np.where(nan, 0, a[0]), np.where(nan, 0, b[0]))
            used = hkv * (d // 2 + d // 16)
            assert np.array_equal(got[:, used:], want[:, used:])
    elif kind == "fp8":                            # a NaN's sign means nothing
        sign = lambda x: np.where(x & 0x7F == 0x7F, 0x7F, x)  # noqa: E731
        assert np.array_equal(sign(got_k), sign(kb)) and np.array_equal(sign(got_v), sign(vb))
    else:
        assert np.array_equal(got_k, kb) and np.array_equal(got_v, vb)
    # keys and values alone, queries in place, another stream: the same bytes
    k2, v2 = _pool(kind, slots, hkv, d, 1), _pool(kind, slots, hkv, d, 2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    td = torch.from_numpy(table).cuda()
    torch.cuda.synchronize()
    sgl.sgl_kv_append(r, params, None, k, v, k2, v2, td, lens, extd, None, ws, stream=s)
    y = qkv.clone()
    yq = y[:, :hq * d].unflatten(1, (hq, d))
    torch.cuda.synchronize()
    assert np.array_equal(_bytes(k2), got_k) and np.array_equal(_bytes(v2), got_v)
    sgl.sgl_kv_append(r, params, yq, k, v, k2, v2, td, lens, extd, yq, ws)
    sgl.sgl_check(ws)
    assert torch.equal(yq[live], qo[live]) and torch.equal(y[:, hq * d:].nan_to_num(), qkv[:, hq * d:].nan_to_num())


@gpu
def test_append_for_many_requests():
    """More requests than one round of the row search takes, most of them without new rows, and four tokens per CTA."""
    rng = np.random.default_rng(3)
    B = 700
    ext = np.where(rng.random(B) < 0.6, 0, rng.integers(0, 25, B))
    rows = int(ext.sum())
    assert rows > 2432
    pre = rng.integers(0, 50, B)
    ld, slots, hkv, d = 80, rows + 10, 2, 64
    table = np.full((B, ld), -1, dtype=np.int32)
    order = rng.permutation(slots)[:rows]
    who = [(r, i) for r in range(B) for i in range(ext[r])]
    for at, (r, i) in enumerate(who):
        table[r, pre[r] + i] = order[at]
    g = torch.Generator().manual_seed(5)
    k, v = (torch.randn(rows + 5, hkv, d, generator=g).bfloat16().cuda() for _ in "kv")
    params = sgl.make_params(sgl.SGL_DTYPE_BF16, B, 2, hkv, d, slots)
    kp, vp = torch.zeros(slots, hkv, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(slots, hkv, d, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    r, freq, amp = _rope(d, d)
    sgl.sgl_kv_append(r, params, None, k, v, kp, vp, torch.from_numpy(table).cuda(),
                      torch.from_numpy(pre.astype(np.int32)).cuda(), torch.from_numpy(ext.astype(np.int32)).cuda(), None, ws)
    sgl.sgl_check(ws)
    pos = np.array([pre[a] + i for a, i in who])
    _check_rotated(kp[order], k[:rows], pos, d, 0, False, freq, amp)
    assert torch.equal(vp[order], v[:rows])
    left = np.setdiff1d(np.arange(slots), order)
    assert not kp[left].any() and not vp[left].any()


@gpu
def test_append_reports_bad_slots_and_positions():
    B, hkv, d, slots, ld = 4, 2, 64, 32, 8
    params = sgl.make_params(sgl.SGL_DTYPE_BF16_FP4KV, B, 4, hkv, d, slots, k_scale=1.0, v_scale=1.0)
    k = torch.ones(B, hkv, d, dtype=torch.bfloat16, device="cuda")
    q = torch.ones(B, 4, d, dtype=torch.bfloat16, device="cuda")
    kp = torch.zeros(slots, fp4.row_bytes(hkv, d), dtype=torch.uint8, device="cuda")
    vp = kp.clone()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    table = torch.arange(B * ld, dtype=torch.int32, device="cuda").view(B, ld)
    table[1, 2], table[2, 0] = slots, -1

    def run(lens):
        kp.zero_()
        qo = torch.zeros_like(q)
        sgl.sgl_kv_append(None, params, q, k, k, kp, vp, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), None,
                          qo, ws)
        return qo
    for lens, wrote, moved in (([1, 3, 2, 0], [0, 17], [1, 1, 1, 0]), ([1, 2, 1, 1], [0, 9, 24], [1, 1, 1, 1]),
                               ([9, 2, 2, 1], [9, 17, 24], [0, 1, 1, 1])):
        qo = run(lens)
        with pytest.raises(sgl.SglError) as e:
            sgl.sgl_check(ws)
        assert e.value.status == -5
        assert kp.any(1).nonzero()[:, 0].tolist() == wrote
        assert qo.any(2).any(1).int().tolist() == moved
    run([1, 2, 2, 0])
    sgl.sgl_check(ws)


@gpu
@pytest.mark.parametrize("decode", [False, True])
def test_mla_append(decode):
    B, H, slots, ld = 5, 16, 200, 60
    rng = np.random.default_rng(4)
    ext = np.ones(B, dtype=np.int64) if decode else np.array([4, 0, 9, 1, 22])
    pre = rng.integers(0, 30, B)
    rows = int(ext.sum())
    who = [(r, i) for r in range(B) for i in range(ext[r])]
    order = rng.permutation(slots)
    table = np.full((B, ld), -1, dtype=np.int32)
    for at, (r, i) in enumerate(who):
        table[r, pre[r] + i] = order[at]
    r, freq, amp = _rope(576, 64, 512, True, "yarn")
    g = torch.Generator().manual_seed(6)
    q = torch.randn(rows, H, 576, generator=g).bfloat16().cuda()
    kv = torch.randn(rows, 576, generator=g).bfloat16().cuda()
    pool = torch.randn(slots, 576, generator=g).bfloat16().cuda()
    old = pool.clone()
    qo = torch.zeros_like(q)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    params = sgl.make_mla_params(B, H, slots)
    sgl.sgl_mla_kv_append(r, params, q, kv, pool, torch.from_numpy(table).cuda(),
                          torch.from_numpy((pre + 1 if decode else pre).astype(np.int32)).cuda(),
                          None if decode else torch.from_numpy(ext.astype(np.int32)).cuda(), qo, ws)
    sgl.sgl_check(ws)
    pos = np.array([pre[a] + i for a, i in who])
    _check_rotated(qo, q, pos, 64, 512, True, freq, amp)
    to = order[:rows]
    _check_rotated(pool[to][:, None], kv[:, None], pos, 64, 512, True, freq, amp)
    left = np.setdiff1d(np.arange(slots), to)
    assert torch.equal(pool[left], old[left])


@gpu
def test_append_in_a_graph_follows_the_lengths():
    """A captured append, replayed after the device lengths have moved on, with other work of the handle in between."""
    B, hkv, d, slots, ld = 3, 2, 128, 64, 16
    r, freq, amp = _rope(d, d)
    params = sgl.make_params(sgl.SGL_DTYPE_BF16, B, 2, hkv, d, slots)
    table = torch.randperm(slots)[:B * ld].view(B, ld).to(torch.int32).cuda()
    k, v = (torch.randn(B, hkv, d, device="cuda").bfloat16() for _ in "kv")
    kp, vp = (torch.zeros(slots, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    lens = torch.tensor([1, 5, 9], dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            sgl.sgl_kv_append(r, params, None, k, v, kp, vp, table, lens, None, None, ws)
    del r
    for _ in range(3):
        kp.zero_()
        graph.replay()
        torch.cuda.synchronize()
        pos = lens.cpu().numpy().astype(np.int64) - 1
        to = table.cpu().numpy()[np.arange(B), pos]
        _check_rotated(kp[to], k, pos, d, 0, False, freq, amp)
        assert int(kp.flatten(1).any(1).sum()) == B
        lens += 1
    sgl.sgl_check(ws)
