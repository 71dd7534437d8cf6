"""The training operators on the GPU against their formulas in 64 bits.

Tolerances, per element, from the arithmetic alone:
* a grouped product is a sum of n products held in fp32 and rounded once:
  |error| <= u |exact| + n 2^-23 sum |a b| (u: half a step of the output type,
  2^-8 bf16, 2^-11 fp16, 2^-24 fp32; the tensor core may truncate, so a whole
  fp32 step per addition);
* SwiGLU: u |exact| plus 2^-18 of the magnitudes that are added (a handful of
  fp32 operations, the exponential's argument is at most ~8 here);
* AdamW: 2^-20 of the magnitudes that are added; codes within one step.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F16, F32, F64 = torch.bfloat16, torch.float16, torch.float32, torch.float64
U = {BF16: 2.0 ** -8, F16: 2.0 ** -11, F32: 2.0 ** -24}
TINY = {BF16: 2.0 ** -133, F16: 2.0 ** -24, F32: 2.0 ** -149}


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


def layout_of(mx, counts, align=1, slack=0):
    """A Layout with the given rows per expert (no routing behind it)."""
    counts = torch.tensor(counts, dtype=torch.int64)
    up = (counts + align - 1) // align * align
    start = up.cumsum(0) - up
    M = max(1, int(up.sum()) + slack)
    i32 = lambda t: t.to(torch.int32).cuda()  # noqa: E731
    return mx.Layout(psum=i32(start + counts), start=i32(start), total=i32(up.sum()[None]),
                     m_indices=i32(torch.empty(0)), src2dst=i32(torch.empty(0, 1)),
                     tile_prefix=i32(torch.empty(0)), E=len(counts), align=align, M_cap=M), \
        list(zip(start.tolist(), (start + counts).tolist()))


def close(got, exact, tol, what):
    bad = (got.double() - exact).abs() > tol
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound, worst "
                           f"{float(((got.double() - exact).abs() / tol.clamp(min=1e-300)).max()):.3g} times")


def product_bound(a, b, exact, dtype):
    """a [i, c], b [j, c] in 64 bits."""
    return U[dtype] * exact.abs() + a.shape[1] * 2.0 ** -23 * (a.abs() @ b.abs().T) + TINY[dtype]


SEGMENTS = {
    "one row": ([1], 1),
    "single rows, empty experts": ([0, 1, 0, 1, 1, 0], 1),
    "ragged": ([5, 0, 129, 64, 1, 300, 0, 17], 1),
    "tile edges": ([128, 256, 127, 257, 64], 1),
    "aligned gaps": ([3, 0, 130, 64, 1], 16),
    "nothing": ([0, 0, 0], 1),
}
SIZES = [(8, 8), (64, 64), (72, 200), (256, 128), (264, 520), (512, 1032)]


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("N,Kd", SIZES)
@pytest.mark.parametrize("seg", SEGMENTS)
def test_products(mx, seg, N, Kd, dtype):
    """All three products of ragged segments, rows outside them poisoned with
    NaN on the way in and untouched on the way out."""
    counts, align = SEGMENTS[seg]
    lay, bounds = layout_of(mx, counts, align, slack=3)
    E, M = lay.E, lay.M_cap
    g = gen(N * 7 + Kd)
    x, dy = normal(g, M, Kd, dtype=dtype), normal(g, M, N, dtype=dtype)
    w = normal(g, E, N, Kd, dtype=dtype, std=0.1)
    inside = torch.zeros(M, dtype=torch.bool, device="cuda")
    for a, b in bounds:
        inside[a:b] = True
    x[~inside] = float("nan")
    dy[~inside] = float("inf")
    y = torch.full((M, N), 7.0, dtype=dtype, device="cuda")
    dx = torch.full((M, Kd), 7.0, dtype=dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert mx.grouped_matmul(x, w, lay, out=y, status=status) is y
    mx.grouped_matmul_dgrad(dy, w, lay, out=dx, status=status)
    dws = {}
    for out in (dtype, F32):
        for acc in (False, True):
            base = normal(gen(3), E, N, Kd, dtype=out)
            dws[out, acc] = base, mx.grouped_matmul_wgrad(dy, x, lay, out=base.clone(), accumulate=acc,
                                                          status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    assert (y[~inside] == 7).all() and (dx[~inside] == 7).all()
    for e, (a, b) in enumerate(bounds):
        X, DY, W = x[a:b].double(), dy[a:b].double(), w[e].double()
        if b > a:
            r = X @ W.T
            close(y[a:b], r, product_bound(X, W, r, dtype), "forward")
            r = DY @ W
            close(dx[a:b], r, product_bound(DY, W.T, r, dtype), "dgrad")
        for (out, acc), (base, got) in dws.items():
            r = DY.T @ X + (base[e].double() if acc else 0)
            tol = product_bound(DY.T, X.T, r, out) if b > a else torch.zeros_like(r)
            if acc:
                tol = tol + 2.0 ** -24 * r.abs()
            close(got[e], r, tol, f"wgrad {out} {acc}")


FEW = {
    "single tokens": [1, 0, 1, 1, 0, 0, 1, 0],
    "a few": [3, 9, 0, 17, 30, 0, 1, 5],
    "one crowded": [0] * 20 + [260] + [0] * 10 + [2],
    "forty": [40, 33, 41, 0, 64, 65, 20, 37],
}


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("N,Kd", [(136, 4104), (1000, 776), (72, 64), (4104, 136)])
@pytest.mark.parametrize("seg", FEW)
def test_few_rows(mx, seg, N, Kd, dtype):
    """Few rows per expert: one and several chunks of rows, contractions whole
    and split over the CTAs of a cluster, in a buffer (align 128) with far more
    rows than pairs."""
    counts = FEW[seg]
    lay, bounds = layout_of(mx, counts, align=128, slack=5)
    lay.src2dst = torch.zeros(sum(counts), 1, dtype=torch.int32, device="cuda")   # one pair per row
    E, M = lay.E, lay.M_cap
    g = gen(N + Kd)
    x, dy = normal(g, M, Kd, dtype=dtype), normal(g, M, N, dtype=dtype)
    w = normal(g, E, N, Kd, dtype=dtype, std=0.1)
    inside = torch.zeros(M, dtype=torch.bool, device="cuda")
    for a, b in bounds:
        inside[a:b] = True
    x[~inside] = float("nan")
    dy[~inside] = float("nan")
    y = torch.full((M, N), 7.0, dtype=dtype, device="cuda")
    dx = torch.full((M, Kd), 7.0, dtype=dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mx.grouped_matmul(x, w, lay, out=y, status=status)
    mx.grouped_matmul_dgrad(dy, w, lay, out=dx, status=status)
    again = mx.grouped_matmul(x, w, lay, out=torch.full_like(y, 7.0))
    torch.cuda.synchronize()
    assert status.item() == 0 and torch.equal(again, y)
    assert (y[~inside] == 7).all() and (dx[~inside] == 7).all()
    for e, (a, b) in enumerate(bounds):
        if b > a:
            X, DY, W = x[a:b].double(), dy[a:b].double(), w[e].double()
            r = X @ W.T
            close(y[a:b], r, product_bound(X, W, r, dtype), "forward")
            r = DY @ W
            close(dx[a:b], r, product_bound(DY, W.T, r, dtype), "dgrad")


def test_weights_of_other_experts_do_not_leak(mx):
    """N and Kd that end inside a tile: the neighbour's infinite and NaN
    weights lie right behind them in memory."""
    lay, bounds = layout_of(mx, [5, 3, 9])
    g = gen(1)
    w = normal(g, 3, 72, 72, dtype=BF16)
    w[0], w[2] = float("nan"), float("inf")
    x = normal(g, lay.M_cap, 72, dtype=BF16)
    a, b = bounds[1]
    for f, ref in ((mx.grouped_matmul, lambda: x[a:b].double() @ w[1].double().T),
                   (mx.grouped_matmul_dgrad, lambda: x[a:b].double() @ w[1].double())):
        got = f(x, w, lay)
        close(got[a:b], ref(), 0.01 * ref().abs() + 0.02, "middle expert")


@pytest.mark.parametrize("E", [1, 33, 160, 1024])
def test_many_experts(mx, E):
    counts = [(e * 7) % 5 for e in range(E)]
    lay, bounds = layout_of(mx, counts)
    g = gen(E)
    x, w = normal(g, lay.M_cap, 64, dtype=BF16), normal(g, E, 40, 64, dtype=BF16)
    dy = normal(g, lay.M_cap, 40, dtype=BF16)
    y, dx = mx.grouped_matmul(x, w, lay), mx.grouped_matmul_dgrad(dy, w, lay)
    dw = mx.grouped_matmul_wgrad(dy, x, lay, out_dtype=F32)
    owner = torch.repeat_interleave(torch.arange(E), torch.tensor(counts)).cuda()
    n = len(owner)
    if n:
        W = w.double()[owner]
        r = torch.einsum("rk,rnk->rn", x[:n].double(), W)
        mag = torch.einsum("rk,rnk->rn", x[:n].double().abs(), W.abs())
        close(y[:n], r, U[BF16] * r.abs() + 64 * 2.0 ** -23 * mag, "forward")
        r = torch.einsum("rn,rnk->rk", dy[:n].double(), W)
        mag = torch.einsum("rn,rnk->rk", dy[:n].double().abs(), W.abs())
        close(dx[:n], r, U[BF16] * r.abs() + 40 * 2.0 ** -23 * mag, "dgrad")
    r = torch.zeros(E, 40, 64, dtype=F64, device="cuda")
    mag = torch.zeros_like(r)
    if n:
        outer = torch.einsum("rn,rk->rnk", dy[:n].double(), x[:n].double())
        r.index_add_(0, owner, outer)
        mag.index_add_(0, owner, outer.abs())
    close(dw, r, 2.0 ** -22 * mag, "wgrad")


@pytest.mark.parametrize("N,Kd,rows", [(768, 2048, 1500), (2048, 768, 700)])
def test_products_of_many_tiles(mx, N, Kd, rows):
    """More tiles than SMs, long contractions, row strides larger than rows."""
    counts = [rows, 3, 0, rows // 2 + 1, 64 * 5]
    lay, bounds = layout_of(mx, counts)
    M, E = lay.M_cap, lay.E
    g = gen(9)
    x = normal(g, M, Kd + 24, dtype=BF16)[:, 8:8 + Kd]
    dy = normal(g, M, N + 8, dtype=BF16)[:, :N]
    w = normal(g, E, N, Kd, dtype=BF16, std=0.05)
    y = torch.zeros(M, N + 16, dtype=BF16, device="cuda")
    mx.grouped_matmul(x, w, lay, out=y[:, 8:8 + N])
    assert (y[:, :8] == 0).all() and (y[:, 8 + N:] == 0).all()
    dx = mx.grouped_matmul_dgrad(dy, w, lay)
    dw = mx.grouped_matmul_wgrad(dy, x, lay)
    for e, (a, b) in enumerate(bounds):
        X, DY, W = x[a:b].double(), dy[a:b].double(), w[e].double()
        r = X @ W.T
        close(y[a:b, 8:8 + N], r, product_bound(X, W, r, BF16), "forward")
        r = DY @ W
        close(dx[a:b], r, product_bound(DY, W.T, r, BF16), "dgrad")
        r = DY.T @ X
        close(dw[e], r, product_bound(DY.T, X.T, r, BF16) if b > a else torch.zeros_like(r), "wgrad")


@pytest.mark.parametrize("mean", [0.0, 0.5])
def test_long_sums_do_not_drift(mx, mean):
    """wgrad over many rows, stored in fp32. The tensor core truncates its
    sums: at most 56 additions (896 rows) of 2^-24 of their size before they
    are added up rounding to nearest. Left alone for all 16384 rows they drift
    by 1.9e-5."""
    g = gen(6)
    lay, bounds = layout_of(mx, [16384, 897, 0, 1793])
    x = (normal(g, lay.M_cap, 264) + mean).to(BF16)
    dy = (normal(g, lay.M_cap, 136) + mean).to(BF16)
    base = normal(g, 4, 136, 264)
    dw = mx.grouped_matmul_wgrad(dy, x, lay, out_dtype=F32)
    added = mx.grouped_matmul_wgrad(dy, x, lay, out=base.clone(), accumulate=True)
    for e, (a, b) in enumerate(bounds):
        r = dy[a:b].double().T @ x[a:b].double()
        bound = 60 * 2.0 ** -24
        assert float((dw[e].double() - r).norm()) <= bound * float(r.norm())
        r = r + base[e].double()
        assert float((added[e].double() - r).norm()) <= bound * float(r.norm())


def test_products_are_repeatable(mx):
    lay, _ = layout_of(mx, [200, 0, 77, 513])
    g = gen(4)
    x, dy = normal(g, lay.M_cap, 512, dtype=BF16), normal(g, lay.M_cap, 264, dtype=BF16)
    w = normal(g, 4, 264, 512, dtype=BF16)
    first = None
    for _ in range(3):
        got = [mx.grouped_matmul(x, w, lay), mx.grouped_matmul_dgrad(dy, w, lay),
               mx.grouped_matmul_wgrad(dy, x, lay, out_dtype=F32)]
        if first is not None:
            assert all(torch.equal(a, b) for a, b in zip(first, got))
        first = got


def test_product_gradients_against_differences(mx):
    """<gradient, d> against the central difference of the loss sum(dy * y)
    along random directions, the loss in 64 bits from the formula."""
    lay, bounds = layout_of(mx, [7, 0, 40, 65])
    g = gen(2)
    x, w = normal(g, lay.M_cap, 72, dtype=F16), normal(g, 4, 136, 72, dtype=F16, std=0.2)
    dy = normal(g, lay.M_cap, 136, dtype=F16)
    dx, dw = mx.grouped_matmul_dgrad(dy, w, lay).double(), mx.grouped_matmul_wgrad(dy, x, lay).double()

    def loss(X, W):
        return sum(float((dy[a:b].double() * (X[a:b] @ W[e].T)).sum()) for e, (a, b) in enumerate(bounds))

    X, W, eps = x.double(), w.double(), 1e-3
    for k in range(4):
        d = normal(gen(50 + k), *x.shape).double()
        want = (loss(X + eps * d, W) - loss(X - eps * d, W)) / (2 * eps)
        tol = float((dx.abs() * d.abs()).sum()) * 2.0 ** -11
        assert abs(float((dx * d).sum()) - want) <= tol
        d = normal(gen(60 + k), *w.shape).double()
        want = (loss(X, W + eps * d) - loss(X, W - eps * d)) / (2 * eps)
        tol = float((dw.abs() * d.abs()).sum()) * 2.0 ** -11
        assert abs(float((dw * d).sum()) - want) <= tol


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("T,K,E,H,align", [(1, 1, 1, 8, 1), (5, 3, 4, 264, 8), (300, 8, 16, 2056, 128),
                                           (64, 2, 8, 512, 32), (1000, 32, 40, 72, 1)])
def test_expand_rows(mx, T, K, E, H, align, dtype):
    g = gen(T)
    ids = torch.rand(T, E, generator=g, device="cuda").topk(K, dim=1).indices.to(torch.int32)
    ids[torch.rand(T, generator=g, device="cuda") < 0.2] = -1
    nv = max(1, T - T // 5)
    n_valid = torch.tensor([nv], dtype=torch.int32, device="cuda")
    M = mx.expanded_capacity(T, K, E, align)
    lay = mx.expand_layout(ids, E, align, M, n_valid)
    x = normal(g, T, H + 8, dtype=dtype)[:, :H]
    x[nv:] = float("nan")
    w = torch.rand(T, K, generator=g, device="cuda")
    out = torch.full((M, H), 5.0, dtype=dtype, device="cuda")
    row_w = torch.full((M,), 5.0, device="cuda")
    mx.expand_rows(x, lay, w, n_valid, out, row_w)
    want, want_w = torch.full_like(out, 5.0), torch.full_like(row_w, 5.0)
    psum = lay.psum.cpu().tolist()
    for e in range(E):
        end = (psum[e] + align - 1) // align * align
        want[psum[e]:end], want_w[psum[e]:end] = 0, 0
    s = lay.src2dst[:nv].long()
    t, k = torch.nonzero(s >= 0, as_tuple=True)
    want[s[t, k]], want_w[s[t, k]] = x[t], w[t, k]
    assert torch.equal(out.view(torch.int16), want.view(torch.int16)) and torch.equal(row_w, want_w)
    # and back: the pairs' values, zero without a pair, padding tokens untouched
    rows = normal(g, M)
    back = torch.full((T, K), 9.0, device="cuda")
    mx.collect_row_grads(rows, lay, n_valid, back)
    expect = torch.where(s >= 0, rows[s.clamp(min=0)], 0.0)
    assert torch.equal(back[:nv], expect) and (back[nv:] == 9).all()


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("M,total,I", [(1, 1, 8), (37, 20, 264), (500, 500, 2048), (3, 0, 64)])
def test_swiglu(mx, M, total, I, dtype):
    lay, _ = layout_of(mx, [total], slack=M - total)
    g = gen(I)
    gu = normal(g, M, 2 * I + 16, dtype=dtype, std=2.0)[:, 8:8 + 2 * I]
    gu[total:] = float("nan")
    if total:
        gu[0, :4] = torch.tensor([0.0, -60.0, 60.0, -0.0], dtype=dtype)
    w = torch.rand(M, generator=g, device="cuda") + 0.1
    dh = normal(g, M, I, dtype=dtype)
    h = torch.full((M, I), 3.0, dtype=dtype, device="cuda")
    dgu = torch.full((M, 2 * I), 3.0, dtype=dtype, device="cuda")
    dr = torch.full((M,), 3.0, device="cuda")
    mx.swiglu(gu, lay, w, out=h)
    mx.swiglu_backward(dh, gu, lay, w, dgu=dgu, drow_w=dr)
    assert (h[total:] == 3).all() and (dgu[total:] == 3).all() and (dr[total:] == 3).all()
    G, V = gu[:total].double().split(I, dim=1)
    W, D = w[:total].double()[:, None], dh[:total].double()
    s = torch.sigmoid(G)
    u, tiny = U[dtype], TINY[dtype]
    r = G * s * V * W
    close(h[:total], r, (u + 2.0 ** -18) * r.abs() + tiny, "h")
    r = D * W * V * s * (1 + G * (1 - s))
    mag = (D * W * V).abs() * s * (1 + (G * (1 - s)).abs())
    close(dgu[:total, :I], r, u * r.abs() + 2.0 ** -18 * mag + tiny, "dg")
    r = D * W * G * s
    close(dgu[:total, I:], r, (u + 2.0 ** -18) * r.abs() + tiny, "du")
    r = (D * G * s * V).sum(1)
    mag = (D * G * s * V).abs().sum(1)
    close(dr[:total], r, (2.0 ** -18 + I * 2.0 ** -24) * mag, "drow_w")
    # without weights, and in place
    h1 = mx.swiglu(gu, lay)
    close(h1[:total], G * s * V, (u + 2.0 ** -18) * (G * s * V).abs() + tiny, "h without weights")
    mine = gu.contiguous()
    mx.swiglu_backward(dh, mine, lay, w, dgu=mine)
    assert torch.equal(mine[:total], dgu[:total])


def test_swiglu_gradient_against_differences(mx):
    M, I = 6, 128
    lay, _ = layout_of(mx, [M])
    g = gen(8)
    gu, dh = normal(g, M, 2 * I, dtype=F16), normal(g, M, I, dtype=F16)
    w = torch.rand(M, generator=g, device="cuda") + 0.5
    dgu, dr = mx.swiglu_backward(dh, gu, lay, w)

    def loss(GU, W):
        G, V = GU.split(I, dim=1)
        return float((dh.double() * (G * torch.sigmoid(G) * V * W[:, None])).sum())

    GU, W, eps = gu.double(), w.double(), 1e-4
    for k in range(4):
        d = normal(gen(70 + k), M, 2 * I).double()
        want = (loss(GU + eps * d, W) - loss(GU - eps * d, W)) / (2 * eps)
        assert abs(float((dgu.double() * d).sum()) - want) <= float((dgu.double() * d).abs().sum()) * 2.0 ** -10
        d = normal(gen(80 + k), M).double()
        want = (loss(GU, W + eps * d) - loss(GU, W - eps * d)) / (2 * eps)
        assert abs(float((dr.double() * d).sum()) - want) <= 1e-5 * float((dr.double() * d).abs().sum()) + 1e-6


# ------------------------------------------------------------------- AdamW
HYPER = dict(lr=2e-3, betas=(0.9, 0.98), eps=1e-8, weight_decay=0.05)


def adamw_formula(p, g, m, v, t, scale, dtype):
    """One step elementwise in `dtype`, an operation at a time."""
    (b1, b2), lr = HYPER["betas"], HYPER["lr"]
    g = g.to(dtype) if scale is None else g.to(dtype) * scale.to(dtype)
    m = m * b1 + g * (1 - b1)
    v = v * b2 + (g * g) * (1 - b2)
    r = v.sqrt()
    step_size, root = lr / (1 - b1 ** t), 1.0 / (1 - b2 ** t) ** 0.5
    p = p.to(dtype) * (1 - lr * HYPER["weight_decay"]) - (m * step_size) / (r * root + HYPER["eps"])
    return p, m, v, r


def to_codes(x, floor):
    n = x.numel()
    b = torch.cat([x, x.new_zeros(-n % 128)]).view(-1, 128)
    amax = b.abs().amax(1, keepdim=True)
    live = amax >= 1e-30
    q = (b * torch.where(live, 448.0 / amax, 0.0)).to(torch.float8_e4m3fn).float()
    if floor:
        q = torch.where((q == 0) & (b > 0) & live, 2.0 ** -9, q)
    q = q.to(torch.float8_e4m3fn).view(torch.uint8).view(-1)[:n]
    return q, torch.where(live, amax * (1.0 / 448.0), 0.0).view(-1)


def from_codes(q, s):
    return q.view(torch.float8_e4m3fn).float() * s.repeat_interleave(128)[: q.numel()]


SHAPES = [(1,), (127,), (128,), (129,), (4096,), (4097,), (33, 65), (3, 5, 7), (0,), (50000,)]


def make_tensors(seed, p_type, g_type, offset):
    """Tensors of odd sizes; offset: storage offsets that break alignment."""
    g = gen(seed)
    ps, gs = [], []
    for s in SHAPES:
        n = int(np.prod(s))
        ps.append(normal(g, n + offset, dtype=p_type)[offset:].view(s))
        gs.append(normal(g, n + offset, dtype=g_type, std=0.01)[offset:].view(s))
    return ps, gs


@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("p_type,g_type,copy", [(F32, BF16, BF16), (F32, F32, None), (BF16, BF16, None),
                                                (F32, F16, F16), (F16, F32, F32)])
def test_adamw(mx, bits, p_type, g_type, copy, offset):
    ps, gs = make_tensors(11, p_type, g_type, offset)
    copies = None if copy is None else [torch.zeros(p.shape, dtype=copy, device="cuda") for p in ps]
    scale = torch.tensor([0.37], device="cuda") if offset else None
    opt = mx.AdamW(ps, state_bits=bits, copies=copies, **HYPER)
    old = [p.clone() for p in ps]
    state = [(torch.zeros(p.numel(), device="cuda"), torch.zeros(p.numel(), device="cuda")) for p in ps]
    for t in range(1, 4):
        gs = [normal(gen(100 * t + i), *g.shape, dtype=g_type, std=0.01 * (1 + i)) for i, g in enumerate(gs)]
        opt.step(gs, grad_scale=scale)
        for i, p in enumerate(ps):
            if p.numel() == 0:
                continue
            m, v = state[i]
            flat = old[i].reshape(-1)
            gi = gs[i].reshape(-1)
            # bit for bit what the formula gives in elementwise fp32
            want, m32, v32, r32 = adamw_formula(flat.float(), gi, m, v, t, scale, F32)
            assert torch.equal(p.reshape(-1), want.to(p_type)), (t, i)
            if copy is not None:
                assert torch.equal(copies[i].reshape(-1), want.to(copy))
            # and near what it gives in 64 bits
            exact, m64, v64, r64 = adamw_formula(flat.double(), gi, m.double(), v.double(), t, scale, F64)
            tol = U[p_type] * exact.abs() + TINY[p_type] + 2.0 ** -20 * (flat.double().abs() + HYPER["lr"] * 10)
            close(p.reshape(-1), exact, tol, "p")
            if bits == 32:
                assert torch.equal(opt.exp_avg[i], m32) and torch.equal(opt.exp_avg_sq[i], v32)
                close(opt.exp_avg[i], m64, 2.0 ** -20 * (m.double().abs() + gi.double().abs()), "m")
                close(opt.exp_avg_sq[i], v64, 2.0 ** -20 * v64, "v")
                state[i] = m32, v32
            else:
                got = []
                for codes, scales, value, floor in ((opt.exp_avg[i], opt.exp_avg_scale[i], m32, False),
                                                    (opt.exp_avg_sq[i], opt.exp_avg_sq_scale[i], r32, True)):
                    q, s = to_codes(value, floor)
                    assert torch.equal(codes, q) and torch.equal(scales, s)
                    back = from_codes(codes, scales)
                    step = (s.repeat_interleave(128)[: q.numel()]) * 2.0 ** -9
                    assert ((back - value).abs() <= torch.maximum(value.abs() / 16, step)).all()
                    got.append(back)
                state[i] = got[0], got[1] * got[1]
            old[i] = p.clone()
    assert opt.steps == 3


def test_adamw_small_root_is_not_lost(mx):
    """One huge gradient beside tiny ones in a block of 128: the tiny ones'
    second moments must not become zero while their first moments live."""
    p = torch.zeros(128, device="cuda")
    g = torch.full((128,), 1e-7, device="cuda")
    g[5] = 1.0
    opt = mx.AdamW([p], state_bits=8, lr=1e-3, weight_decay=0.0)
    for _ in range(3):
        opt.step([g])
    assert (opt.exp_avg_sq[0] != 0).all()
    assert p.abs().max() < 4e-3
    # nothing but zeros stays zeros
    z = torch.zeros(300, device="cuda")
    opt = mx.AdamW([z], state_bits=8, weight_decay=0.0)
    opt.step([torch.zeros(300, device="cuda")])
    assert (z == 0).all() and (opt.exp_avg_scale[0] == 0).all() and (opt.exp_avg_sq[0] == 0).all()


@pytest.mark.parametrize("count", [1, 16, 17, 400, 401, 1000])
@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_many_tensors(mx, bits, count):
    g = gen(count)
    sizes = [1 + (i * 37) % 300 for i in range(count)]
    ps = [normal(g, n) for n in sizes]
    gs = [normal(g, n, std=0.1) for n in sizes]
    old = [p.clone() for p in ps]
    mx.AdamW(ps, state_bits=bits, **HYPER).step(gs)
    for p, o, gi in zip(ps, old, gs):
        z = torch.zeros_like(o)
        assert torch.equal(p, adamw_formula(o, gi, z, z, 1, None, F32)[0])


def test_adamw_goes_on_from_a_checkpoint(mx):
    ps, gs = make_tensors(3, F32, F32, 0)
    again = [p.clone() for p in ps]
    for bits in (32, 8):
        a = mx.AdamW(ps, state_bits=bits, **HYPER)
        a.step(gs)
        b = mx.AdamW([p.copy_(q) for p, q in zip(again, ps)], state_bits=bits, step=a.steps, **HYPER,
                     exp_avg=[t.clone() for t in a.exp_avg], exp_avg_sq=[t.clone() for t in a.exp_avg_sq],
                     exp_avg_scale=[t.clone() for t in a.exp_avg_scale] or None,
                     exp_avg_sq_scale=[t.clone() for t in a.exp_avg_sq_scale] or None)
        a.step(gs)
        b.step(gs)
        assert all(torch.equal(x, y) for x, y in zip(ps, again))
        assert all(torch.equal(x, y) for x, y in zip(a.exp_avg_sq, b.exp_avg_sq))


def test_adamw_follows_new_storage(mx):
    p, g = normal(gen(1), 500), normal(gen(2), 500)
    opt = mx.AdamW([p], weight_decay=0.0)
    opt.step([g])
    before = p.data
    p.data = p.data.clone()
    kept = before.clone()
    opt.step([g])
    assert torch.equal(before, kept) and not torch.equal(p, kept)


# --------------------------------------------------------------- the layer
@pytest.mark.parametrize("T,K,E,H,I,align,nv", [(1, 2, 4, 64, 64, 1, 1), (96, 2, 6, 384, 128, 8, 96),
                                                (200, 4, 8, 256, 520, 128, 150), (64, 8, 160, 72, 40, 1, 64)])
def test_layer_against_autograd(mx, T, K, E, H, I, align, nv):
    """TrainableExperts' output and gradients against autograd of the layer's
    formula in 64 bits on the same bf16 inputs. Every intermediate is rounded
    to bf16 once (2^-8 at most), four roundings deep: 2 % of the result's norm."""
    g = gen(T)
    w13 = normal(g, E, 2 * I, H, dtype=BF16, std=H ** -0.5)
    w2 = normal(g, E, H, I, dtype=BF16, std=I ** -0.5)
    x, dy = normal(g, T, H, dtype=BF16), normal(g, T, H, dtype=BF16)
    ids = torch.rand(T, E, generator=g, device="cuda").topk(K, dim=1).indices.to(torch.int32)
    if T > 10:
        ids[3] = -1
        ids[5, 0] = -1
    w = torch.rand(T, K, generator=g, device="cuda")
    n_valid = torch.tensor([nv], dtype=torch.int32, device="cuda")
    layer = mx.TrainableExperts(w13, w2, K=K, max_tokens=T, align=align)
    y = layer.forward(x, ids, w, n_valid)
    y = y.clone()
    dx, dw = layer.backward(dy)
    dx, dtw = dx.clone(), dw.clone()
    grads = [t.clone() for t in layer.gradients]
    torch.cuda.synchronize()
    assert layer.status.item() == 0
    X, W = x[:nv].double().requires_grad_(), w[:nv].double().requires_grad_()
    W13, W2 = w13.double().requires_grad_(), w2.double().requires_grad_()
    out = torch.zeros(nv, H, dtype=F64, device="cuda")
    for e in range(E):
        t, k = torch.nonzero(ids[:nv] == e, as_tuple=True)
        if len(t):
            G, V = (X[t] @ W13[e].T).split(I, dim=1)
            out = out.index_add(0, t, W[t, k][:, None] * ((torch.nn.functional.silu(G) * V) @ W2[e].T))
    out.backward(dy[:nv].double())

    def near(got, want, what):
        fro = float((got.double() - want).norm() / want.norm().clamp(min=1e-300))
        assert fro <= 0.02, (what, fro)

    near(y[:nv], out.detach(), "y")
    near(dx[:nv], X.grad, "dx")
    near(dtw[:nv], torch.where(ids[:nv] >= 0, W.grad, 0), "dtopk_w")
    near(grads[0], W13.grad, "dw13")
    near(grads[1], W2.grad, "dw2")
    # a second micro-batch adds to the weights' gradients
    layer.forward(x, ids, w, n_valid)
    layer.backward(dy, accumulate=True)
    for a, b in zip(layer.gradients, grads):
        assert torch.equal(a, b + b)
    with pytest.raises(RuntimeError):
        layer.backward(dy)


def test_wrong_bound_on_rows_is_flagged(mx):
    """A layout that says it has three pairs, with segments of 200 rows: the
    rows the few-rows form leaves out are not left out silently."""
    lay, _ = layout_of(mx, [200, 0, 0, 0])
    lay.src2dst = torch.zeros(3, 1, dtype=torch.int32, device="cuda")
    w, x = normal(gen(1), 4, 64, 64, dtype=BF16), normal(gen(2), lay.M_cap, 64, dtype=BF16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mx.grouped_matmul(x, w, lay, status=status)
    assert status.item() == -5   # MOE_ERR_DEVICE_CHECK


def test_nothing_to_do(mx):
    """No tokens, no rows, no parameters; a single row with any stride."""
    lay, _ = layout_of(mx, [0, 0])
    lay.M_cap = 0
    w = normal(gen(1), 2, 64, 72, dtype=BF16)
    x, dy = w.new_zeros(0, 72), w.new_zeros(0, 64)
    assert mx.grouped_matmul(x, w, lay).shape == (0, 64)
    assert mx.grouped_matmul_dgrad(dy, w, lay).shape == (0, 72)
    assert (mx.grouped_matmul_wgrad(dy, x, lay, out=torch.ones(2, 64, 72, device="cuda")) == 0).all()
    kept = mx.grouped_matmul_wgrad(dy, x, lay, out=torch.ones(2, 64, 72, device="cuda"), accumulate=True)
    assert (kept == 1).all()
    assert mx.swiglu(dy, lay).shape == (0, 32)
    dgu, dr = mx.swiglu_backward(dy[:, :32], dy, lay)
    assert dgu.shape == (0, 64) and dr.shape == (0,)
    lay.src2dst = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    assert mx.expand_rows(x, lay).shape == (0, 72)
    assert mx.collect_row_grads(torch.zeros(0, device="cuda"), lay).shape == (0, 2)
    opt = mx.AdamW([])
    opt.step([])
    assert opt.steps == 1
    lay, _ = layout_of(mx, [0, 1])
    row = normal(gen(2), 1, 75, dtype=BF16)[:, :72]
    r = row.double() @ w[1].double().T
    close(mx.grouped_matmul(row, w, lay), r, product_bound(row.double(), w[1].double(), r, BF16), "one row")
    torch.cuda.synchronize()


def test_capture(mx):
    """A forward, backward and step recorded into a CUDA graph and replayed."""
    g = gen(9)
    T, K, E, H, I = 64, 2, 4, 128, 64
    layer = mx.TrainableExperts(normal(g, E, 2 * I, H, dtype=BF16, std=0.1),
                                normal(g, E, H, I, dtype=BF16, std=0.1), K=K, max_tokens=T)
    x, dy = normal(g, T, H, dtype=BF16), normal(g, T, H, dtype=BF16)
    w, ids = torch.rand(T, E, generator=g, device="cuda").topk(K, dim=1)
    ids, w = ids.to(torch.int32).contiguous(), w.contiguous()

    def step(stream=None):
        y = layer.forward(x, ids, w, stream=stream)
        dx, dw = layer.backward(dy, stream=stream)
        return y, dx, dw, *layer.gradients

    want = [t.clone() for t in step()]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            got = step(side)
    for t in got:
        t.zero_()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_other_stream(mx):
    """Calls queued on a stream of their own, behind work that makes their
    inputs there."""
    lay, bounds = layout_of(mx, [130, 7])
    g = gen(5)
    w = normal(g, 2, 256, 128, dtype=BF16)
    src = normal(g, lay.M_cap, 128, dtype=BF16)
    want = mx.grouped_matmul(src, w, lay)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    x, out = torch.zeros_like(src), torch.zeros_like(want)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        x.copy_(src)
        mx.grouped_matmul(x, w, lay, out=out)
    mx.grouped_matmul(src, w, lay, stream=s)
    s.synchronize()
    assert torch.equal(out, want)


def test_python_refusals(mx):
    lay, _ = layout_of(mx, [4, 4])
    x = torch.zeros(8, 64, dtype=BF16, device="cuda")
    w = torch.zeros(2, 64, 64, dtype=BF16, device="cuda")
    with pytest.raises(ValueError):
        mx.grouped_matmul(x.float(), w, lay)
    with pytest.raises(ValueError):
        mx.grouped_matmul(x, w.half(), lay)
    with pytest.raises(ValueError):
        mx.grouped_matmul(x, w[:1], lay)
    with pytest.raises(ValueError):
        mx.grouped_matmul(x.t(), w, lay)
    with pytest.raises(ValueError):
        mx.grouped_matmul(x, w, lay, out=torch.zeros(8, 56, dtype=BF16, device="cuda"))
    with pytest.raises(mx.MoEError):
        mx.grouped_matmul(x[:, :60], torch.zeros(2, 64, 60, dtype=BF16, device="cuda"), lay)
    with pytest.raises(ValueError):
        mx.grouped_matmul_wgrad(x, x, lay, accumulate=True)
    with pytest.raises(ValueError):
        mx.grouped_matmul_wgrad(x, x, lay, out=torch.zeros(2, 64, 64, dtype=F16, device="cuda"))
    with pytest.raises(ValueError):
        mx.swiglu(x, lay, row_w=torch.zeros(7, device="cuda"))
    with pytest.raises(ValueError):
        mx.expand_rows(x.float(), lay)
    with pytest.raises(ValueError):
        mx.AdamW([x.t()])
    with pytest.raises(ValueError):
        mx.AdamW([x], state_bits=4)
    opt = mx.AdamW([x])
    with pytest.raises(ValueError):
        opt.step([])
    with pytest.raises(ValueError):
        opt.step([torch.zeros(7, device="cuda")])
    with pytest.raises(ValueError):
        opt.step([x], grad_scale=torch.zeros(2, device="cuda"))
    assert opt.steps == 0


@pytest.mark.parametrize("bits", [32, 8])
def test_example_learns(mx, bits):
    """The example's layer approaches its teacher: the loss falls to under half."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "train_experts.py")
    spec = importlib.util.spec_from_file_location("train_experts", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    losses = m.main(["--steps", "80", "--state-bits", str(bits)])
    assert all(np.isfinite(losses))
    assert np.mean(losses[-5:]) < 0.5 * np.mean(losses[:5]), (losses[:5], losses[-5:])


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("N,Kd", [(64, 72), (200, 520), (512, 512)])
@pytest.mark.parametrize("counts", [[2000], [777, 0, 1, 5003], [64 * 40, 64 * 8 + 1]],
                         ids=["one", "uneven", "whole blocks"])
def test_wgrad_of_few_tiles_over_many_rows(mx, counts, N, Kd, dtype):
    """Few tiles, long sums: the rows are shared by the CTAs of a cluster, some
    of which have none for a small expert."""
    lay, bounds = layout_of(mx, counts, slack=2)
    M, E = lay.M_cap, lay.E
    g = gen(N + Kd)
    x, dy = normal(g, M, Kd + 8, dtype=dtype)[:, :Kd], normal(g, M, N, dtype=dtype)
    x[bounds[-1][1]:] = float("nan")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for out in (dtype, F32):
        for acc in (False, True):
            base = normal(gen(3), E, N, Kd, dtype=out)
            got = mx.grouped_matmul_wgrad(dy, x, lay, out=base.clone(), accumulate=acc, status=status)
            again = mx.grouped_matmul_wgrad(dy, x, lay, out=base.clone(), accumulate=acc)
            assert torch.equal(got, again)
            for e, (a, b) in enumerate(bounds):
                X, DY = x[a:b].double(), dy[a:b].double()
                r = DY.T @ X + (base[e].double() if acc else 0)
                tol = product_bound(DY.T, X.T, r, out) if b > a else torch.zeros_like(r)
                if acc:
                    tol = tol + 2.0 ** -24 * r.abs()
                close(got[e], r, tol, f"wgrad {out} {acc}")
    assert status.item() == 0


@pytest.mark.parametrize("counts", [[50000], [9000, 3, 0, 40, 6000]], ids=["eight parts", "four parts"])
def test_wgrad_in_parts(mx, counts):
    """More parts than the smaller experts have blocks of rows."""
    lay, bounds = layout_of(mx, counts)
    g = gen(12)
    x, dy = normal(g, lay.M_cap, 200, dtype=BF16), normal(g, lay.M_cap, 136, dtype=BF16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for out in (BF16, F32):
        for acc in (False, True):
            base = normal(gen(3), lay.E, 136, 200, dtype=out)
            got = mx.grouped_matmul_wgrad(dy, x, lay, out=base.clone(), accumulate=acc, status=status)
            for e, (a, b) in enumerate(bounds):
                r = dy[a:b].double().T @ x[a:b].double() + (base[e].double() if acc else 0)
                # chunks of 896 rows, or 4096 for 16-bit results, then the parts
                drift = (60 if out is F32 else 260) * 2.0 ** -24
                bound = (drift + (U[out] if out is BF16 else 0)) * float(r.norm())
                assert float((got[e].double() - r).norm()) <= bound, (out, acc, e)
    assert status.item() == 0
