"""Chunk calls whose device lengths are others than the host copies that planned them: shorter ones are followed, longer
ones are reported and leave the scores of requests without room as they were."""

import numpy as np
import pytest
import torch

import radixattention_prefix_shared_radix_gb300 as sgl
from tests.test_gpu_attn_weights import KINDS, Cache, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from radixattention_prefix_shared_radix_gb300 import build
    build.build()


class Planned:
    """Rows of a table 2000 wide; a call planned for some lengths and run with others."""

    def __init__(self, kind, pre, ext, window=0):
        self.c = Cache(kind, np.full(len(pre), 2000), 8, 2, 64, seed=3)
        self.pre, self.ext, self.window = np.array(pre), np.array(ext), window
        self.q = self.c.queries(int(self.ext.sum()))
        self.lse = 5 + torch.randn(len(self.q), 8, generator=torch.Generator().manual_seed(4))
        self.p = self.c.params(host_prefix_lens=self.pre, host_extend_lens=self.ext)
        self.ws = torch.zeros(sgl.sgl_attn_weights_workspace_bytes(self.p, window), dtype=torch.uint8, device="cuda")
        self.dev = [x.cuda() for x in (self.q, self.lse, self.c.pool, torch.from_numpy(self.c.table))]

    def run(self, pre, ext):
        out = torch.full((len(pre), 2000), 7.0, device="cuda")
        d = [torch.from_numpy(np.asarray(x, dtype=np.int32)).cuda() for x in (pre, ext)]
        sgl.sgl_attn_weights(*self.dev, *d, self.p, None, out, self.ws, window=self.window)
        return out.cpu().numpy()

    def alone(self, pre, ext):
        """The same with what was planned for these lengths."""
        pre, ext = np.asarray(pre), np.asarray(ext)
        n = int(ext.sum())
        return _run(self.c, self.q[:n], self.lse[:n], pre, ext, self.window, None, 1.0, False)


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("window", [0, 7])
def test_a_prefix_longer_than_planned(kind, window):
    x = Planned(kind, [100, 300, 50], [40, 20, 30], window)
    want = x.alone(x.pre, x.ext)
    assert np.array_equal(x.run(x.pre, x.ext), want)
    sgl.sgl_check(x.ws)
    for longer in (1500, 1980):
        got = x.run([100, longer, 50], x.ext)
        with pytest.raises(sgl.SglError) as e:
            sgl.sgl_check(x.ws)
        assert e.value.status == -5
        assert np.array_equal(got[0], want[0]) and (got[1] == 7).all()
        assert np.array_equal(got[2], want[2]) or (got[2] == 7).all()
    assert np.array_equal(x.run(x.pre, x.ext), want)
    sgl.sgl_check(x.ws)


@pytest.mark.parametrize("kind", list(KINDS))
def test_many_prefixes_longer_than_planned(kind):
    """What was planned for 70 requests of a tile each has room for a few of eight tiles: every row gets the weights of its
    length, or nothing."""
    x = Planned(kind, [60] * 70, [2] * 70)
    longer = [60] + [1990] * 67 + [60] * 2
    want = x.alone(longer, x.ext)
    got = x.run(longer, x.ext)
    with pytest.raises(sgl.SglError):
        sgl.sgl_check(x.ws)
    assert np.array_equal(got[0], want[0])
    left = [bool((got[r] == 7).all()) for r in range(70)]
    # (runs of one query block in both plans: the same bits)
    assert all(left[r] or np.array_equal(got[r], want[r]) for r in range(70)) and all(left[9:68])


@pytest.mark.parametrize("kind", list(KINDS))
def test_shorter_lengths_are_followed(kind):
    x = Planned(kind, [700, 300, 50], [90, 20, 300])
    for pre, ext in (([10, 300, 50], [90, 20, 300]), ([700, 0, 3], [1, 0, 299]), ([0, 0, 0], [0, 0, 0])):
        got = x.run(pre, ext)
        sgl.sgl_check(x.ws)
        L = np.add(pre, ext)
        if not sum(ext):
            assert (got == 7).all()
            continue
        want = x.alone(pre, ext)
        for r in range(3):
            # (other runs, other orders of addition: 2^-24 for each of at most 2400 weights)
            assert np.allclose(got[r, :L[r]], want[r, :L[r]], rtol=2400 * 2.0 ** -24, atol=0)
            assert (got[r, L[r]:] == 7).all()


@pytest.mark.parametrize("kind", ["bf16", "fp4"])
def test_a_captured_chunk_reports_lengths_without_room(kind):
    x = Planned(kind, [100, 300], [40, 20])
    want = x.alone(x.pre, x.ext)
    d = [torch.from_numpy(y.astype(np.int32)).cuda() for y in (x.pre, x.ext)]
    out = torch.full((2, 2000), 7.0, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            sgl.sgl_attn_weights(*x.dev, *d, x.p, None, out, x.ws)
    for pre, fits in ((300, True), (1900, False), (300, True)):
        out.fill_(7.0)
        d[0][1] = pre
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = out.cpu().numpy()
        assert np.array_equal(got[0], want[0])
        if fits:
            sgl.sgl_check(x.ws)
            assert np.array_equal(got[1], want[1])
        else:
            assert (got[1] == 7).all()
            with pytest.raises(sgl.SglError):
                sgl.sgl_check(x.ws)
