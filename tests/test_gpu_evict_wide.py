"""Short requests in a slot table much wider than they are: scores no wider than the longest request bound the call."""

import numpy as np
import pytest

import radixattention_prefix_shared_radix_gb300 as sgl
from tests.test_gpu_evict import Rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from radixattention_prefix_shared_radix_gb300 import build
    build.build()


@pytest.mark.parametrize("ld", [8193, 131072, 140000, 900000])
@pytest.mark.parametrize("page", [1, 16])
@pytest.mark.parametrize("in_place", [False, True])
def test_narrow_scores_over_a_wide_table(ld, page, in_place):
    lens = [0, 1, 17, 2000, 2048, 333]
    r = Rows(lens, [n // 2 for n in lens], "spread", ld=ld, sld=2048, seed=ld)
    r.check(page, 4, 32, in_place)


@pytest.mark.parametrize("ld", [8193, 40000, 131072, 140000])
@pytest.mark.parametrize("page", [1, 16])
@pytest.mark.parametrize("in_place", [False, True])
def test_short_rows_in_wide_tables(ld, page, in_place):
    lens = [0, 1, 15, 16, 17, 100, 1000, 2048, 8192]
    r = Rows(lens, [n // 3 for n in lens], "ties", ld=ld, sld=ld, seed=ld)
    r.check(page, 4, 32, in_place)


def test_a_request_longer_than_its_scores_is_reported():
    r = Rows([2050, 30], [10, 10], "spread", ld=140000, sld=2048)
    (s, t, p, n), ev, cnt, ws = r.run()
    with pytest.raises(sgl.SglError) as e:
        sgl.sgl_check(ws)
    assert e.value.status == -5 and n.tolist() == [10, 10] and cnt.tolist() == [2038, 20]
    assert (t[0, 2048:] == 77).all() and (ev[:, 2038:] == 99).all()
    assert np.array_equal(np.sort(np.concatenate([t[0, :10], ev[0, :2038]])), np.sort(r.table[0, :2048]))
