"""What a mask hides has no part in a result: values of later tokens in an extend over a cache."""

import numpy as np
import pytest
import torch

from tests.test_gpu_fp4 import _own
from tests.test_gpu_nan import Run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from radixattention_prefix_shared_radix_gb300 import build
    build.build()


@pytest.mark.parametrize("kind", ["f32", "fp4"])
@pytest.mark.parametrize("hq,hkv,d", [(16, 4, 64), (32, 8, 128), (8, 1, 128), (9, 9, 64)])
def test_extend_over_a_nan_value_reaches_no_earlier_token(kind, hq, hkv, d):
    """A token does not see the values of later ones, not even through a product with a weight of zero."""
    pre, ext = np.array([0, 150, 30]), np.array([300, 170, 1])
    r = Run(kind, _own(list(pre + ext)), hq, hkv, d, seed=5)
    b, G, n = r.b, hq // hkv, int(ext.sum())
    g = torch.Generator().manual_seed(6)
    q = torch.randn(n, hq, d, generator=g).to(r.q.dtype)
    clean = r.extend(r.k, r.v, pre, ext, q)
    who = [(x, int(pre[x]) + i) for x in range(3) for i in range(ext[x])]
    for marks in ([(0, 0)], [(0, 77)], [(0, 299)], [(1, 20)], [(1, 150)], [(1, 151)], [(1, 200), (1, 319)], [(2, 30)],
                  [(0, 127), (0, 128), (1, 160), (2, 3)]):
        v, hit = r.v, np.zeros((n, hq, d), dtype=bool)
        for at, (req, pos) in enumerate(marks):
            h, e = (hkv - 1 + at) % hkv, (17 + 32 * at) % d
            v = r.nan(v, b.table[req, pos], h, e)
            cols = slice(e // 16 * 16, e // 16 * 16 + 16) if kind == "fp4" else e
            for i, (x, p) in enumerate(who):
                if x == req and p >= pos:
                    hit[i, h * G:(h + 1) * G, cols] = True
        o, lse = r.extend(r.k, v, pre, ext, q)
        hit = torch.as_tensor(hit)
        assert o[hit].isnan().all()
        assert torch.equal(o[~hit], clean[0][~hit]) and torch.equal(lse, clean[1])
