"""Sines and cosines of the rotation, each relative to its own size.

With b = 0 a rotated pair is (a cos t, a sin t).  Sine and cosine are fp32 values within one unit in the last place
(2^-23 of themselves), the product and the amplitude's share round once each (2^-24): together under 2^-22 of the
result.  The angle is the position times the frequency as a double; the library holds it as a fraction of a turn, off by
2^-64 turns per position, and the reference's product rounds it by 2^-53: under 2^-51 of the angle together, which
matters only next to a zero of the function.
"""

import numpy as np
import pytest
import torch

import radixattention_prefix_shared_radix_gb300 as sgl
from oracle import rope as orope

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from radixattention_prefix_shared_radix_gb300 import build
    build.build()


def _angles(d, theta, pos, kind=sgl.SGL_ROPE_SCALE_NONE, **kw):
    """(cosines, sines [n, d / 2]) that the library rotates by, and the float64 angles."""
    r = sgl.sgl_rope_create(d, theta=theta, scaling=kind, **kw)
    x = torch.zeros(len(pos), 1, d, device="cuda")
    x[..., :d // 2] = 1.0
    sgl.sgl_rope(r, x, None, torch.tensor(pos, dtype=torch.int32, device="cuda"))
    y = x[:, 0].double().cpu().numpy()
    name = {sgl.SGL_ROPE_SCALE_NONE: "none", sgl.SGL_ROPE_SCALE_LINEAR: "linear", sgl.SGL_ROPE_SCALE_NTK: "ntk"}[kind]
    t = np.asarray(pos, dtype=np.float64)[:, None] * orope.frequencies(d, theta, name, **kw)
    return y[:, :d // 2], y[:, d // 2:], t


@pytest.mark.parametrize("d,theta,kind,kw", [
    (128, 1e4, sgl.SGL_ROPE_SCALE_NONE, {}), (128, 1e6, sgl.SGL_ROPE_SCALE_NONE, {}),
    (128, 5e5, sgl.SGL_ROPE_SCALE_LINEAR, dict(factor=4.0)), (64, 1e8, sgl.SGL_ROPE_SCALE_NTK, dict(factor=8.0))])
def test_small_and_nearly_whole_turns(d, theta, kind, kw):
    pos = list(range(0, 800)) + [1420, 2130, 4096, 33102, 103993, 104348, 131071]
    c, s, t = _angles(d, theta, pos, kind, **kw)
    for got, want in ((c, np.cos(t)), (s, np.sin(t))):
        err, tol = np.abs(got - want), 2.0 ** -22 * np.abs(want) + 2.0 ** -51 * t
        assert (err <= tol).all(), "worst %.3g of the bound" % (err / np.maximum(tol, 1e-300)).max()


def test_far_positions():
    """At the farthest positions the angle of pair 0 (frequency one) is that of the position itself."""
    pos = [2 ** 31 - 1 - i for i in range(50)] + [2 ** 30 + 17 * i for i in range(50)] + [2 ** 24 + i for i in range(9)]
    c, s, t = _angles(64, 10000.0, pos)
    for got, want in ((c, np.cos(t)), (s, np.sin(t))):
        # (pair 0: its angle is exact in float64, and in the library off by 2^-64 turns per position)
        err, tol = np.abs(got - want)[:, 0], (2.0 ** -22 * np.abs(want) + 2.0 ** -62 * t)[:, 0]
        assert (err <= tol).all(), "worst %.3g of the bound" % (err / tol).max()
        err, tol = np.abs(got - want), 2.0 ** -22 * np.abs(want) + 2.0 ** -51 * t
        assert (err <= tol).all(), "worst %.3g of the bound" % (err / tol).max()
