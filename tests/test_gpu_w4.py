"""The experts' product over 4-bit weights on the GPU against its formula in 64
bits.

Tolerance: a code less its zero point is exact in 16 bits, a product with x exact
in fp32; a sum of n of them in the tensor core (which may truncate: 2^-23 of the
magnitudes per addition), a product with the scale and an addition per group,
partial sums; and one rounding of the result (u):
  |error| <= u |exact| + (n + 16) 2^-23 sum |x w|.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F16, F32, F64 = torch.bfloat16, torch.float16, torch.float32, torch.float64
U = {BF16: 2.0 ** -8, F16: 2.0 ** -11}
TINY = {BF16: 2.0 ** -133, F16: 2.0 ** -24}
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def mx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from expanded_layout_expert_gb300 import build
    build.build()
    import expanded_layout_expert_gb300 as m
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, dtype=F32, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def layout_of(mx, counts, align=1, slack=0, pairs=None):
    """A Layout with the given rows per expert; pairs: rows that src2dst allows
    for (none: the buffer's)."""
    counts = torch.tensor(counts, dtype=torch.int64)
    up = (counts + align - 1) // align * align
    start = up.cumsum(0) - up
    M = max(1, int(up.sum()) + slack)
    i32 = lambda t: t.to(torch.int32).cuda()  # noqa: E731
    return mx.Layout(psum=i32(start + counts), start=i32(start), total=i32(up.sum()[None]),
                     m_indices=i32(torch.empty(0)), src2dst=i32(torch.empty(pairs or 0, 1)),
                     tile_prefix=i32(torch.empty(0)), E=len(counts), align=align, M_cap=M), \
        list(zip(start.tolist(), (start + counts).tolist()))


def weights(g, E, N, Kd, group, dtype, zeros):
    codes = torch.randint(0, 256, (E, N, Kd // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = (torch.rand(E, N, Kd // group, generator=g, device="cuda") * 0.1 + 0.01).to(dtype)
    z = torch.randint(0, 16, (E, N, Kd // group), generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    return codes, scales, z


def dense(codes, scales, z, e):
    """Expert e's weights in 64 bits."""
    q = torch.stack([codes[e] & 15, codes[e] >> 4], dim=2).flatten(1).double()
    group = q.shape[1] // scales.shape[2]
    off = 8.0 if z is None else z[e].double().repeat_interleave(group, 1)
    return (q - off) * scales[e].double().repeat_interleave(group, 1)


def check(mx, counts, N, Kd, group, dtype, zeros, align=1, slack=3, pairs=None, seed=0):
    lay, bounds = layout_of(mx, counts, align, slack, pairs)
    E, M = lay.E, lay.M_cap
    g = gen(seed + N * 7 + Kd)
    x = normal(g, M, Kd + 8, dtype=dtype)[:, :Kd]
    codes, scales, z = weights(g, E, N, Kd, group, dtype, zeros)
    inside = torch.zeros(M, dtype=torch.bool, device="cuda")
    for a, b in bounds:
        inside[a:b] = True
    x[~inside] = NAN
    out = torch.full((M, N + 16), 7.0, dtype=dtype, device="cuda")[:, 8:N + 8]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert mx.grouped_matmul_w4(x, codes, scales, lay, zeros=z, out=out, status=status) is out
    torch.cuda.synchronize()
    assert status.item() == 0
    assert (out[~inside] == 7).all()
    for e, (a, b) in enumerate(bounds):
        if b == a:
            continue
        X, W = x[a:b].double(), dense(codes, scales, z, e)
        exact = X @ W.T
        tol = U[dtype] * exact.abs() + (Kd + 16) * 2.0 ** -23 * (X.abs() @ W.abs().T) + TINY[dtype]
        bad = ~((out[a:b].double() - exact).abs() <= tol)
        assert not bad.any(), (e, int(bad.sum()), torch.nonzero(bad)[0].tolist())


SEGMENTS = {
    "one row": ([1], 1),
    "single rows, empty experts": ([0, 1, 0, 1, 1, 0], 1),
    "few": ([3, 9, 0, 17, 30, 0, 1, 5], 1),
    "eights": ([8, 16, 32, 7, 15, 31, 33, 64], 1),
    "ragged": ([5, 0, 129, 64, 1, 300, 0, 17], 1),
    "aligned gaps": ([3, 0, 130, 64, 1], 16),
    "nothing": ([0, 0, 0], 1),
}
SIZES = [(8, 32, 32), (64, 64, 64), (72, 96, 32), (136, 128, 128), (64, 192, 64), (200, 1152, 128), (264, 544, 32),
         (520, 1088, 64), (1032, 2048, 128)]


@pytest.mark.parametrize("zeros", [False, True], ids=["", "zeros"])
@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("N,Kd,group", SIZES)
@pytest.mark.parametrize("seg", SEGMENTS)
def test_product(mx, seg, N, Kd, group, dtype, zeros):
    counts, align = SEGMENTS[seg]
    check(mx, counts, N, Kd, group, dtype, zeros, align)


@pytest.mark.parametrize("rows", [1, 8, 9, 16, 17, 24, 33, 63, 65, 100, 129])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_rows_of_one_expert(mx, rows, group):
    check(mx, [0, rows, 2], 328, 640, group, BF16, True, seed=rows)


# rows of six experts, with more weights than the form for few rows takes: tiles of
# 16, 32, 48 and 64 rows, one and several of them, and experts without rows
CROWDS = {"16": [10, 0, 3, 40, 1, 6], "32": [16, 33, 0, 17, 30, 9],
          "48": [48, 33, 97, 0, 19, 13], "64": [64, 5, 130, 0, 65, 31]}


@pytest.mark.parametrize("zeros", [False, True], ids=["", "zeros"])
@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("N,Kd,group", [(1096, 1952, 32), (1032, 2048, 32), (1160, 1984, 64), (1288, 1728, 64),
                                        (1024, 2176, 128), (1296, 2304, 128)])
@pytest.mark.parametrize("rows", CROWDS)
def test_more_rows(mx, rows, N, Kd, group, dtype, zeros):
    """Sizes that end inside tiles, stages and steps."""
    counts = CROWDS[rows]
    mean = -(-sum(counts) // len(counts))
    tile = "16" if mean <= 12 else "32" if mean <= 26 else "48" if mean <= 40 else "64"
    assert len(counts) * N * Kd > 1 << 23 and tile == rows
    check(mx, counts, N, Kd, group, dtype, zeros, align=8, slack=2, pairs=sum(counts), seed=len(rows))


@pytest.mark.parametrize("group", [32, 64, 128])
def test_contractions_split_over_a_cluster(mx, group):
    """Few tiles and a long contraction: several CTAs a tile."""
    check(mx, [40], 264, 8192, group, BF16, True, pairs=40)
    check(mx, [33, 12], 128, 16384 + 128, group, F16, False, pairs=45)
    check(mx, [200], 72, 4096, group, BF16, True, pairs=200)


def test_single_tokens_over_long_contractions(mx):
    """The form for few rows: scales of a row that are whole vectors in shared
    memory, and not; more of them than it takes."""
    for Kd, group in ((4096, 32), (4096 + 32, 32), (6528, 64), (7168, 128), (7168 - 128, 128)):
        check(mx, [1, 0, 2, 8, 1], 200, Kd, group, BF16, True, pairs=12)
    check(mx, [1, 3], 40, 65536, 32, F16, True, pairs=4)


def test_long_contraction_and_many_experts(mx):
    check(mx, [2, 0, 40], 72, 16384, 128, BF16, True)
    check(mx, [i % 3 for i in range(1024)], 16, 64, 32, F16, False)
    check(mx, [0] * 1000 + [1, 0, 70] + [0] * 21, 40, 256, 64, BF16, True, pairs=71)


def test_buffer_larger_than_the_pairs(mx):
    """The grid goes by the pairs there may be, the buffer has many more rows."""
    check(mx, [3, 1, 0, 12], 136, 256, 128, BF16, False, align=128, slack=500, pairs=16)
    lay, _ = layout_of(mx, [40, 40], pairs=10)   # a wrong bound on the rows is said
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    codes, scales, _ = weights(gen(0), 2, 64, 64, 64, BF16, False)
    mx.grouped_matmul_w4(normal(gen(1), 80, 64, dtype=BF16), codes, scales, lay, status=status)
    assert status.item() == -5


def test_zero_points_use_four_bits_and_default_to_eight(mx):
    lay, _ = layout_of(mx, [4, 5])
    g = gen(3)
    x = normal(g, 9, 256, dtype=F16)
    codes, scales, z = weights(g, 2, 64, 256, 128, F16, True)
    y = mx.grouped_matmul_w4(x, codes, scales, lay, zeros=z)
    assert torch.equal(y, mx.grouped_matmul_w4(x, codes, scales, lay, zeros=z + 0x50))
    eight = torch.full_like(z, 8)
    assert torch.equal(mx.grouped_matmul_w4(x, codes, scales, lay),
                       mx.grouped_matmul_w4(x, codes, scales, lay, zeros=eight))


def test_values_that_are_not_finite_stay_in_their_rows_and_columns(mx):
    lay, _ = layout_of(mx, [6, 40])
    g = gen(5)
    x = normal(g, 46, 384, dtype=BF16)
    codes, scales, z = weights(g, 2, 72, 384, 128, BF16, True)
    clean = mx.grouped_matmul_w4(x, codes, scales, lay, zeros=z)
    x2, s2 = x.clone(), scales.clone()
    x2[2, 100], x2[20, 0], s2[1, 17, 2] = NAN, INF, INF
    y = mx.grouped_matmul_w4(x2, codes, s2, lay, zeros=z)
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[2], hit[20], hit[6:, 17] = True, True, True
    assert not y[hit].isfinite().any()
    assert torch.equal(y[~hit], clean[~hit])


def test_results_do_not_change_from_run_to_run(mx):
    lay, _ = layout_of(mx, [1, 0, 30, 100, 7])
    g = gen(5)
    x = normal(g, 138, 2048, dtype=BF16)
    codes, scales, z = weights(g, 5, 520, 2048, 64, BF16, True)
    first = mx.grouped_matmul_w4(x, codes, scales, lay, zeros=z)
    for _ in range(5):
        assert torch.equal(first, mx.grouped_matmul_w4(x, codes, scales, lay, zeros=z))


def test_many_experts_with_more_rows(mx):
    check(mx, [i % 21 for i in range(1024)], 136, 96, 32, BF16, True, pairs=sum(i % 21 for i in range(1024)))
    check(mx, [0] * 500 + [70, 0, 31] + [0] * 521, 264, 128, 128, F16, False, pairs=101)


@pytest.mark.parametrize("rows", [3, 40])
def test_offsets_past_32_bits(mx, rows):
    """Codes of 2.3 GB, with rows at the first and the last expert."""
    E, N, Kd, group = 160, 4096, 7168, 128
    counts = [rows] + [0] * (E - 2) + [rows]
    lay, bounds = layout_of(mx, counts, pairs=2 * rows)
    g = gen(rows)
    x = normal(g, 2 * rows, Kd, dtype=BF16)
    codes, scales, z = weights(g, E, N, Kd, group, BF16, True)
    out = mx.grouped_matmul_w4(x, codes, scales, lay, zeros=z)
    for e in (0, E - 1):
        a, b = bounds[e]
        X, W = x[a:b].double(), dense(codes, scales, z, e)
        exact = X @ W.T
        tol = U[BF16] * exact.abs() + (Kd + 16) * 2.0 ** -23 * (X.abs() @ W.abs().T)
        assert ((out[a:b].double() - exact).abs() <= tol).all(), e


def test_not_finite_in_tiles_of_more_rows(mx):
    """Rows of x past the chunk's in its tile, other experts' weights in the tile of
    weight rows, scales and rows that are not finite."""
    counts = [40, 33, 61]
    lay, _ = layout_of(mx, counts, pairs=sum(counts))
    g = gen(6)
    x = normal(g, sum(counts), 2048, dtype=BF16)
    codes, scales, z = weights(g, 3, 1480, 2048, 128, BF16, True)
    clean = mx.grouped_matmul_w4(x, codes, scales, lay, zeros=z)
    x2, s2 = x.clone(), scales.clone()
    x2[40], x2[70, 100], s2[1, 1479, 2], s2[2, 0, 0] = NAN, INF, INF, NAN
    y = mx.grouped_matmul_w4(x2, codes, s2, lay, zeros=z)
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[40], hit[70], hit[40:73, 1479], hit[73:, 0] = True, True, True, True
    assert not y[hit].isfinite().any()
    assert torch.equal(y[~hit], clean[~hit])


def test_more_rows_than_said_are_flagged(mx):
    """A wrong bound on the rows, in the form for more of them."""
    lay, _ = layout_of(mx, [200, 300], pairs=100)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    codes, scales, _ = weights(gen(0), 2, 64, 64, 64, BF16, False)
    mx.grouped_matmul_w4(normal(gen(1), 500, 64, dtype=BF16), codes, scales, lay, status=status)
    assert status.item() == -5


def test_calls_on_two_streams_at_once(mx):
    """Both forms share nothing between calls."""
    g = gen(9)
    cases = []
    for counts, pairs in (([1, 2, 0, 1], 4), ([40, 50, 3, 64], 157)):
        lay, _ = layout_of(mx, counts, pairs=pairs)
        x = normal(g, sum(counts), 1024, dtype=BF16)
        w = weights(g, 4, 1032, 1024, 64, BF16, True)
        cases.append((x, w, lay, mx.grouped_matmul_w4(x, w[0], w[1], lay, zeros=w[2])))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = []
    for i in range(40):
        x, w, lay, want = cases[i % 2]
        s = streams[i % 4]
        got.append((mx.grouped_matmul_w4(x, w[0], w[1], lay, zeros=w[2], stream=s), want))
    torch.cuda.synchronize()
    for a, b in got:
        assert torch.equal(a, b)
