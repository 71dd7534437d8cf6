"""A wait of the 4-bit product that runs out: the library's own test call leaves
one copy out and waits a few milliseconds for it. The status says so, the tile is
not stored, the others are, and the next call is as ever."""
import time

import pytest
import torch

from test_gpu_w4 import BF16, dense, gen, layout_of, mx, normal, weights  # noqa: F401

pytestmark = pytest.mark.gpu

LIMIT = 10_000_000   # cycles: some 5 ms
TIMEOUT = -6
KEPT = 7.0


class Case:
    def __init__(self, mx, counts, N, Kd, pairs):  # noqa: F811
        self.mx, self.N, self.Kd, self.pairs = mx, N, Kd, pairs
        self.lay, self.bounds = layout_of(mx, counts, pairs=pairs)
        g = gen(N + Kd)
        self.x = normal(g, self.lay.M_cap, Kd, dtype=BF16)
        self.codes, self.scales, self.z = weights(g, len(counts), N, Kd, 128, BF16, True)

    def run(self, cta, block):
        """(out, status) without the copy of `block` for `cta`."""
        out = torch.full((self.lay.M_cap, self.N), KEPT, dtype=BF16, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        lay = self.lay
        self.mx.check(self.mx.load().moe_selftest_w4_wait(
            self.x.data_ptr(), self.Kd, self.codes.data_ptr(), self.scales.data_ptr(), self.z.data_ptr(),
            lay.start.data_ptr(), lay.psum.data_ptr(), lay.E, self.N, self.Kd, lay.M_cap, self.pairs,
            out.data_ptr(), self.N, LIMIT, cta, block, status.data_ptr(),
            torch.cuda.current_stream().cuda_stream), "moe_selftest_w4_wait")
        torch.cuda.synchronize()
        return out, status.item()

    def whole(self):
        """The result with every copy made, held against the formula."""
        out, status = self.run(-1, 0)
        assert status == 0
        for e, (a, b) in enumerate(self.bounds):
            X, W = self.x[a:b].double(), dense(self.codes, self.scales, self.z, e)
            exact = X @ W.T
            tol = 2.0 ** -8 * exact.abs() + (self.Kd + 16) * 2.0 ** -23 * (X.abs() @ W.abs().T)
            assert ((out[a:b].double() - exact).abs() <= tol).all()
        return out


# 40 rows and 5 of two experts are three chunks; 520 columns three tiles, of whose last
# the second warpgroup has none; 896 contracted values seven stages in a ring of four
@pytest.fixture(scope="module")
def case(mx):  # noqa: F811
    c = Case(mx, [40, 5], 520, 896, 45)
    return c, c.whole()


@pytest.mark.parametrize("block", range(7))
@pytest.mark.parametrize("cta,rows,columns", [(0, (0, 32), (0, 256)), (4, (32, 40), (256, 512)),
                                              (8, (40, 45), (512, 520))])
def test_a_copy_that_does_not_come(case, cta, rows, columns, block):
    c, want = case
    t0 = time.perf_counter()
    out, status = c.run(cta, block)
    assert status == TIMEOUT
    assert time.perf_counter() - t0 < 1.0   # what waits for something never asked for takes 2 s
    lost = torch.zeros_like(out, dtype=torch.bool)
    lost[rows[0]:rows[1], columns[0]:columns[1]] = True
    assert (out[lost] == KEPT).all()
    assert torch.equal(out[~lost], want[~lost])
    again, status = c.run(-1, 0)
    assert status == 0 and torch.equal(again, want)


def test_a_block_that_there_is_not(case):
    c, want = case
    for cta, block in ((0, 7), (9, 0), (1 << 30, 3)):
        out, status = c.run(cta, block)
        assert status == 0 and torch.equal(out, want)


@pytest.fixture(scope="module")
def shared(mx):  # noqa: F811
    """Contractions of 64 stages split over the eight CTAs of a cluster: three chunks
    of rows, two tiles of columns."""
    c = Case(mx, [40, 12], 264, 8192, 52)
    return c, c.whole()


@pytest.mark.parametrize("rank", [0, 3, 7])
@pytest.mark.parametrize("tile,rows,columns", [(0, (0, 32), (0, 256)), (3, (32, 40), (256, 264)),
                                               (4, (40, 52), (0, 256))])
@pytest.mark.parametrize("block", [0, 5])
def test_no_one_of_the_cluster_stores(shared, tile, rows, columns, rank, block):
    """The others of a cluster have their own sums, but not the tile's."""
    c, want = shared
    out, status = c.run(tile * 8 + rank, block)
    assert status == TIMEOUT
    lost = torch.zeros_like(out, dtype=torch.bool)
    lost[rows[0]:rows[1], columns[0]:columns[1]] = True
    assert (out[lost] == KEPT).all()
    assert torch.equal(out[~lost], want[~lost])
    again, status = c.run(-1, 0)
    assert status == 0 and torch.equal(again, want)
