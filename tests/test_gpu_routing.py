"""The router, the weighted return of rows and their gradients on the GPU,
against their formulas in 64 bits.

Tolerances, from the arithmetic alone (one fp32 rounding: 2^-24 of the value; u:
half a step of the output type):
* a weight: e^x with its argument rounded is within (|x| + 3) 2^-24, a sum of E
  of them in E / 32 + 5 additions, a quotient; together (|x| + E / 32 + 24) 2^-24
  of the value, x being the logit's distance from the one it is held against;
* a logit's gradient: u of the value, and (|x| + E / 32 + 64) 2^-24 of the
  magnitudes that are added;
* combine: u of the value, and 2^-24 per term, twice, of the magnitudes added;
* its row gradient: u, and one product's rounding; its weight gradient: H
  products and additions, 2^-24 of the magnitudes each.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F16, F32, F64 = torch.bfloat16, torch.float16, torch.float32, torch.float64
U = {BF16: 2.0 ** -8, F16: 2.0 ** -11, F32: 2.0 ** -24}
TINY = {BF16: 2.0 ** -133, F16: 2.0 ** -24, F32: 2.0 ** -149}
INF, NAN = float("inf"), float("nan")


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


def close(got, exact, tol, what):
    got = got.double()
    same = (got == exact) | (got.isnan() & exact.isnan())
    bad = ~same & ~((got - exact).abs() <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound, first at "
                           f"{torch.nonzero(bad)[0].tolist()}: {got[bad][0]} for {exact[bad][0]}")


# ------------------------------------------------------------------ router
def special_rows(logits, K):
    """Ties, experts that may not be chosen, fewer than K, none, huge values."""
    T, E = logits.shape
    rows = [torch.zeros(E), torch.full((E,), -INF), torch.full((E,), -3.0), torch.arange(E) * -0.25]
    few = torch.full((E,), -INF)
    few[E // 2:E // 2 + max(1, K // 2)] = 1.5
    signed = torch.zeros(E)
    signed[::2] = -0.0
    steep = torch.linspace(-3e4, 3e4, E) if E > 1 else torch.tensor([3e4])
    low = torch.full((E,), -200.0)
    low[-1] = -190.0
    rows += [few, signed, steep, low, torch.full((E,), NAN)]
    one_nan = torch.zeros(E)
    one_nan[0] = NAN
    rows += [one_nan]
    rows = torch.stack(rows)[:T].to(logits)
    logits[:len(rows)] = rows
    return logits


def chosen(logits, bias, K):
    key = logits.float() if bias is None else logits.float() + bias
    key = torch.where(key.isnan(), torch.full_like(key, -INF), key)
    order = key.cpu().sort(dim=1, descending=True, stable=True)
    ids = order.indices[:, :K].to(logits.device)
    return torch.where(key.gather(1, ids) > -INF, ids, -1)


def weights64(l, ids, score, renormalize, factor):
    """topk_w in 64 bits, differentiable in l [T, E]."""
    ok = ids >= 0
    lk = torch.where(ok, l.gather(1, ids.clamp(min=0)), -INF)
    if score == "softmax":
        if renormalize:
            top = lk.detach().amax(1, keepdim=True)
            z = torch.where(ok, (lk - top).exp(), 0.0)
            w = torch.where(ok, z / z.sum(1, keepdim=True), 0.0)
        else:
            dead = (l.detach() == -INF).all(1, keepdim=True)
            w = torch.where(ok, torch.softmax(torch.where(dead, 0.0, l), 1).gather(1, ids.clamp(min=0)), 0.0)
    else:
        # log s, so that quotients of tiny scores keep their digits
        logs = torch.nn.functional.logsigmoid(torch.where(ok, lk, 0.0))
        if renormalize:
            top = torch.where(ok, logs, -INF).detach().amax(1, keepdim=True)
            z = torch.where(ok, (logs - top).exp(), 0.0)
            w = torch.where(ok, z / z.sum(1, keepdim=True), 0.0)
        else:
            w = torch.where(ok, logs.exp(), 0.0)
    return factor * w


def distance(l, ids, score, renormalize):
    """|x| of the exponentials behind each weight."""
    lk = l.gather(1, ids.clamp(min=0))
    if score == "sigmoid" and not renormalize:
        return lk.abs()
    held = l if not renormalize else torch.where(ids >= 0, lk, -INF)
    top = torch.where(held.isnan(), -INF, held).amax(1, keepdim=True)
    d = (lk - top).abs() + (lk.abs() if score == "sigmoid" else 0.0)
    return torch.nan_to_num(d, nan=0.0, posinf=0.0)


SHAPES = [(1, 1), (2, 2), (8, 2), (33, 5), (64, 8), (100, 1), (160, 8), (257, 32), (1024, 32)]


@pytest.mark.parametrize("biased", [False, True], ids=["", "bias"])
@pytest.mark.parametrize("renormalize", [False, True], ids=["", "renorm"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=["f32", "bf16", "fp16"])
@pytest.mark.parametrize("E,K", SHAPES)
def test_route(mx, E, K, dtype, score, renormalize, biased):
    check_route(mx, 41, E, K, dtype, score, renormalize, biased)


@pytest.mark.parametrize("score,renormalize", [("softmax", False), ("sigmoid", True)])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("E,K", [(1, 1), (8, 2), (15, 4), (31, 8), (48, 6), (64, 8), (65, 8), (96, 1), (97, 8), (128, 7),
                                 (129, 8), (160, 8), (161, 8), (192, 8), (193, 8), (256, 8), (64, 9), (512, 8), (768, 3)])
def test_route_rows_for_eight_lanes(mx, E, K, dtype, score, renormalize):
    """Rows enough for the forms in which a warp takes four at a time, a last part of a warp's among them."""
    check_route(mx, 20001, E, K, dtype, score, renormalize, E % 2 == 0)


def check_route(mx, T, E, K, dtype, score, renormalize, biased):
    factor = 2.5
    g = gen(E * 5 + K)
    wide = normal(g, T, E + 3, dtype=dtype, std=2.0)
    logits = wide[:, 1:E + 1]   # a stride, and an address that fits the type alone
    special_rows(logits, K)
    bias = normal(g, E) if biased else None
    ids, w = mx.route_topk(logits, K, score=score, renormalize=renormalize, factor=factor, bias=bias)
    want = chosen(logits, bias, K)
    assert torch.equal(ids.long(), want)
    l = logits.double()
    exact = weights64(l, want, score, renormalize, factor)
    x = distance(l, want, score, renormalize)
    close(w, exact, (x + E / 32 + 24) * 2.0 ** -24 * exact.abs() + factor * 2.0 ** -126, "weights")
    assert (w[want < 0] == 0).all()

    # gradient: against the formula's, by differentiation in 64 bits
    dw = normal(g, T, K)
    dl = mx.route_topk_backward(dw, logits, ids, score=score, renormalize=renormalize, factor=factor)
    assert dl.dtype is dtype
    l = l.clone().requires_grad_()
    fine = ~l.detach().isnan().any(1)
    y = weights64(torch.where(fine[:, None] & l.isfinite(), l, -1e300), want, score, renormalize, factor)
    y = torch.where(fine[:, None], y, 0.0)
    (y * dw.double()).sum().backward()
    exact = torch.nan_to_num(l.grad)
    size = torch.zeros_like(exact)   # of what is added
    wabs = torch.nan_to_num(weights64(l.detach(), want, score, renormalize, 1.0))
    g_abs = torch.where(want >= 0, factor * dw.double().abs(), 0.0)
    size.scatter_add_(1, want.clamp(min=0), wabs * (g_abs + (g_abs * wabs).sum(1, keepdim=True)))
    if score == "softmax" and not renormalize:
        p = torch.nan_to_num(torch.softmax(l.detach(), 1))
        size += p * (g_abs * wabs).sum(1, keepdim=True)
    # e^x of a difference |x| from the largest logit: at most 88, beyond it is 0
    x = 90.0
    tol = U[dtype] * exact.abs() + (x + E / 32 + 64) * 2.0 ** -24 * size + TINY[dtype] + factor * 2.0 ** -120
    close(dl[fine], exact[fine], tol[fine], "gradient")


@pytest.mark.parametrize("score,renormalize", [("softmax", False), ("softmax", True), ("sigmoid", False),
                                               ("sigmoid", True)])
def test_route_gradient_against_differences(mx, score, renormalize):
    T, E, K, h = 6, 11, 3, 1e-5
    g = gen(2)
    logits, dw = normal(g, T, E, std=1.5), normal(g, T, K)
    ids, _ = mx.route_topk(logits, K, score=score, renormalize=renormalize)
    dl = mx.route_topk_backward(dw, logits, ids, score=score, renormalize=renormalize)
    for e in range(E):
        d = torch.zeros(T, E, dtype=F64, device="cuda")
        d[:, e] = h
        f = [(weights64(logits.double() + s * d, ids.long(), score, renormalize, 1.0) * dw.double()).sum(1)
             for s in (1, -1)]
        slope = (f[0] - f[1]) / (2 * h)
        # h^2 / 6 of a third derivative of at most ~10, 1e-16 / h of the difference, fp32's roundings
        assert ((dl[:, e].double() - slope).abs() <= 2e-9 + 1e-10 + 1e-5 * dw.double().abs().sum(1)).all()


def test_route_valid_rows_and_given_buffers(mx):
    T, E, K = 9, 12, 4
    logits = normal(gen(1), T, E)
    logits[5:] = NAN
    nv = torch.tensor([5], dtype=torch.int32, device="cuda")
    ids = torch.full((T, K), 77, dtype=torch.int32, device="cuda")
    w = torch.full((T, K), 7.0, device="cuda")
    assert mx.route_topk(logits, K, n_valid=nv, ids=ids, weights=w)[0] is ids
    assert (ids[5:] == 77).all() and (w[5:] == 7).all() and (ids[:5] >= 0).all()
    made_ids, made_w = mx.route_topk(logits, K, n_valid=nv)
    assert torch.equal(made_ids[:5], ids[:5]) and (made_ids[5:] == -1).all() and (made_w[5:] == 0).all()
    dl = torch.full((T, E), 7.0, device="cuda")
    mx.route_topk_backward(torch.ones(T, K, device="cuda"), logits, ids, n_valid=nv, out=dl)
    assert (dl[5:] == 7).all() and dl[:5].isfinite().all() and (dl[:5] != 7).all()
    for bad in (0, -3, 100):   # a count out of range is clamped
        nv.fill_(bad)
        mx.route_topk(logits[:5].contiguous(), K, n_valid=nv)
    assert mx.route_topk(logits[:0], K)[0].shape == (0, K)
    mx.route_topk_backward(torch.ones(0, K, device="cuda"), logits[:0], ids[:0])


def test_route_gradient_of_ids_that_repeat_or_are_none(mx):
    """An expert that comes twice adds twice; ids outside [0, E) are no pairs."""
    T, E, K = 3, 7, 4
    logits, dw = normal(gen(4), T, E), normal(gen(5), T, K)
    ids = torch.tensor([[2, 2, 5, -1], [6, 6, 6, 6], [-1, 9, 1, 2 ** 30]], dtype=torch.int32, device="cuda")
    for score in ("softmax", "sigmoid"):
        for renormalize in (False, True):
            dl = mx.route_topk_backward(dw, logits, ids, score=score, renormalize=renormalize)
            l = logits.double().requires_grad_()
            k = torch.where((ids >= 0) & (ids < E), ids, -1).long()
            w = weights64(l, k, score, renormalize, 1.0)
            (w * dw.double()).sum().backward()
            close(dl, l.grad, torch.full_like(l, 90 * 2.0 ** -24 * 16), f"{score} {renormalize}")


def test_route_many_rows(mx):
    """More rows than the grid has warps at a time."""
    T, E, K = 100003, 40, 6
    logits = normal(gen(8), T, E, dtype=BF16)   # plenty of ties
    ids, w = mx.route_topk(logits, K)
    assert torch.equal(ids.long(), chosen(logits, None, K))
    close(w, weights64(logits.double(), ids.long(), "softmax", False, 1.0), 64 * 2.0 ** -24 * w.double(), "weights")


# ------------------------------------------------------------------ weighted return
def pairs(mx, T, K, E, align, seed, inactive=0.2, n_valid=None):
    """A layout made by the library from random ids (some tokens without any)."""
    g = gen(seed)
    ids = torch.rand(T, E, generator=g, device="cuda").argsort(1)[:, :K].to(torch.int32)
    if K > E:
        ids = torch.randint(0, E, (T, K), generator=g, device="cuda", dtype=torch.int32)
    ids[torch.rand(T, generator=g, device="cuda") < inactive] = -1
    ids[torch.rand(T, K, generator=g, device="cuda") < 0.1] = -1
    M = mx.expanded_capacity(T, K, E, align) + 5
    return mx.expand_layout(ids.contiguous(), E, align, M, n_valid)


COMBINE = [(1, 8, 1, 2, 1), (3, 72, 2, 4, 1), (37, 264, 7, 9, 8), (50, 1032, 8, 16, 16), (21, 2056, 9, 12, 128),
           (5, 7168, 32, 3, 1), (300, 128, 3, 5, 1)]


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("weighted", [True, False], ids=["w", "plain"])
@pytest.mark.parametrize("residual", ["none", "given", "in place"])
@pytest.mark.parametrize("T,H,K,E,align", COMBINE)
def test_combine_rows(mx, T, H, K, E, align, residual, weighted, dtype):
    lay = pairs(mx, T, K, E, align, seed=T * 3 + H)
    src = lay.src2dst.long()
    g = gen(H + K)
    rows = normal(g, lay.M_cap, H + 16, dtype=dtype)[:, 8:H + 8]
    used = torch.zeros(lay.M_cap, dtype=torch.bool, device="cuda")
    used[src[src >= 0]] = True
    rows[~used] = NAN
    w = None
    if weighted:
        w = normal(g, T, K)
        w[src < 0] = INF   # of no pair: not used
    res = None if residual == "none" else normal(g, T, H + 8, dtype=dtype)[:, :H]
    exact = torch.zeros(T, H, dtype=F64, device="cuda") if res is None else res.double()
    size = exact.abs()
    for k in range(K):
        t = torch.nonzero(src[:, k] >= 0)[:, 0]
        term = rows[src[t, k]].double() * (w[t, k, None].double() if weighted else 1.0)
        exact = exact.index_add(0, t, term)
        size = size.index_add(0, t, term.abs())
    out = res if residual == "in place" else torch.full((T, H + 24), 7.0, dtype=dtype, device="cuda")[:, :H]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert mx.combine_rows(rows, lay, w, residual=res, out=out, status=status) is out
    assert status.item() == 0
    close(out, exact, U[dtype] * exact.abs() + 2 * (K + 1) * 2.0 ** -24 * size + TINY[dtype], "combine")


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("weighted", [True, False], ids=["w", "plain"])
@pytest.mark.parametrize("in_place", [False, True], ids=["", "in place"])
@pytest.mark.parametrize("T,H,K,E,align", COMBINE + [(5000, 264, 2, 6, 16), (701, 1032, 9, 16, 8), (450, 4104, 2, 6, 1)])
def test_combine_rows_backward(mx, T, H, K, E, align, in_place, weighted, dtype):
    lay = pairs(mx, T, K, E, align, seed=T * 3 + H)
    src = lay.src2dst.long()
    g = gen(H + K + 1)
    rows = normal(g, lay.M_cap, H + 8, dtype=dtype)[:, :H]
    used = torch.zeros(lay.M_cap, dtype=torch.bool, device="cuda")
    used[src[src >= 0]] = True
    rows[~used] = NAN
    dy = normal(g, T, H + 8, dtype=dtype)[:, 8:]
    w = None
    if weighted:
        w = normal(g, T, K)
        w[src < 0] = NAN
    before = rows.clone()
    drows = rows if in_place else torch.full((lay.M_cap, H), 7.0, dtype=dtype, device="cuda")
    old = drows.clone()
    got, dw = mx.combine_rows_backward(dy, rows, lay, w, drows=drows)
    assert got is drows
    gap = torch.zeros_like(used)   # aligned segments' ends, zeroed
    for a, b in zip(lay.start.tolist(), lay.psum.tolist()):
        gap[b:(b + align - 1) // align * align] = True
    assert (drows[gap] == 0).all()
    other = ~gap & ~used
    assert torch.equal(drows[other].nan_to_num(5.0), old[other].nan_to_num(5.0))
    for k in range(K):
        t = torch.nonzero(src[:, k] >= 0)[:, 0]
        r, d = src[t, k], dy[t].double()
        exact = d * (w[t, k, None].double() if weighted else 1.0)
        close(drows[r], exact, (U[dtype] + 2.0 ** -23) * exact.abs() + TINY[dtype], "drows")
        terms = d * before[r].double()
        close(dw[t, k], terms.sum(1), (H + 8) * 2.0 ** -24 * terms.abs().sum(1) + 1e-37, "dtopk_w")
    assert (dw[src < 0] == 0).all()


def test_combine_gradient_against_differences(mx):
    """sum(dy * combine(rows, w)) moved along random directions of rows and w:
    the form is bilinear, so the central difference has no error of its own but
    the results' rounding (u of each of T H values)."""
    T, H, K, E = 12, 64, 3, 5
    lay = pairs(mx, T, K, E, 4, seed=1)
    g = gen(9)
    rows, dy, w = normal(g, lay.M_cap, H, dtype=BF16), normal(g, T, H, dtype=BF16), normal(g, T, K)
    drows, dw = mx.combine_rows_backward(dy, rows, lay, w)
    size = 0.0
    for what in ("rows", "w"):
        v = torch.randint(-1, 2, (rows if what == "rows" else w).shape, generator=g, device="cuda").float()
        f = []
        for s in (0.5, -0.5):   # exact steps of bf16 values would need rows on a grid: take them in w, 64-bit rows
            if what == "w":
                y = mx.combine_rows(rows, lay, w + s * v)
                size = y.double().abs()
            else:
                moved = (rows.float() + s * v).bfloat16()
                y = mx.combine_rows(moved, lay, w)
                size = y.double().abs()
            f.append((y.double() * dy.double()).sum())
        if what == "w":
            slope = (dw.double() * v.double()).sum()
            slack = 0.0
        else:
            step = (rows.float() + 0.5 * v).bfloat16().double() - (rows.float() - 0.5 * v).bfloat16().double()
            used = torch.zeros(lay.M_cap, 1, dtype=F64, device="cuda")
            used[lay.src2dst[lay.src2dst >= 0].long()] = 1
            slope = (drows.double() * step * used).sum()
            slack = 2.0 ** -8 * (drows.double() * step * used).abs().sum()
        tol = 2 * 2.0 ** -8 * (size * dy.double().abs()).sum() + slack
        assert abs((f[0] - f[1]) - slope) <= 1.5 * tol


def test_combine_valid_rows_and_rows_out_of_range(mx):
    T, H, K, E = 10, 40, 2, 4
    nv = torch.tensor([6], dtype=torch.int32, device="cuda")
    lay = pairs(mx, T, K, E, 1, seed=3, inactive=0.0)
    rows, w = normal(gen(1), lay.M_cap, H, dtype=F16), normal(gen(2), T, K)
    out = torch.full((T, H), 7.0, dtype=F16, device="cuda")
    mx.combine_rows(rows, lay, w, n_valid=nv, out=out)
    assert (out[6:] == 7).all() and (out[:6] != 7).any()
    drows, dw = torch.full_like(rows, 7.0), torch.full((T, K), 7.0, device="cuda")
    mx.combine_rows_backward(normal(gen(3), T, H, dtype=F16), rows, lay, w, n_valid=nv, drows=drows, dtopk_w=dw)
    late = lay.src2dst[6:][lay.src2dst[6:] >= 0].long()
    assert (dw[6:] == 7).all() and (drows[late] == 7).all()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lay.src2dst[0, 0] = lay.M_cap   # behind the last row: skipped, and said
    mx.combine_rows(rows, lay, w, status=status)
    assert status.item() == -5
    status.zero_()
    _, dw = mx.combine_rows_backward(normal(gen(3), T, H, dtype=F16), rows, lay, w, status=status)
    assert status.item() == -5 and dw[0, 0] == 0


def test_router_and_return_on_other_streams_and_captured(mx):
    """Calls queued behind a busy stream, and a captured chain of all four that
    is replayed on other inputs."""
    T, H, K, E = 64, 256, 4, 16
    M = mx.expanded_capacity(T, K, E, 1)
    g = gen(6)
    logits, x, dy = normal(g, T, E), normal(g, T, H, dtype=BF16), normal(g, T, H, dtype=BF16)

    def chain():
        ids, w = mx.route_topk(logits, K, renormalize=True)
        lay = mx.expand_layout(ids, E, 1, M)
        rows = mx.expand_rows(x, lay)
        y = mx.combine_rows(rows, lay, w, residual=x)
        drows, dw = mx.combine_rows_backward(dy, rows, lay, w)
        return [ids, w, y, drows, dw, mx.route_topk_backward(dw, logits, ids, renormalize=True)]

    want = chain()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        got = chain()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = chain()
    for seed in (7, 8):
        logits.copy_(normal(gen(seed), T, E))
        x.copy_(normal(gen(seed + 10), T, H))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, chain()):
            assert torch.equal(a, b)
    # the weights sum to one: the return of the tokens' own rows doubles them
    close(held[2], 2 * x.double(), (2.0 ** -8 + 1e-6) * 2 * x.double().abs(), "return")


def test_offsets_past_32_bits(mx):
    """Rows of 4.6 GB: the last ones go back to tokens, and get their gradients."""
    M, H, T, K = 320_000, 7168, 3, 2
    rows = torch.zeros(M, H, dtype=BF16, device="cuda")
    src = torch.tensor([[0, M - 1], [M - 2, 1], [-1, M - 3]], dtype=torch.int32, device="cuda")
    used = src[src >= 0].long()
    g = gen(2)
    rows[used] = normal(g, len(used), H, dtype=BF16)
    one = torch.full((1,), M, dtype=torch.int32, device="cuda")
    lay = mx.Layout(psum=one, start=torch.zeros_like(one), total=one, m_indices=one[:0], src2dst=src,
                    tile_prefix=one[:0], E=1, align=1, M_cap=M)
    w, dy = normal(g, T, K), normal(g, T, H, dtype=BF16)
    out = mx.combine_rows(rows, lay, w)
    drows, dw = mx.combine_rows_backward(dy, rows, lay, w)
    for t in range(T):
        exact, size = torch.zeros(H, dtype=F64, device="cuda"), 0
        for k in range(K):
            r = int(src[t, k])
            if r < 0:
                assert dw[t, k] == 0
                continue
            term = rows[r].double() * w[t, k].double()
            exact, size = exact + term, size + term.abs()
            close(drows[r], dy[t].double() * w[t, k].double(),
                  (2.0 ** -8 + 2.0 ** -23) * (dy[t].double() * w[t, k].double()).abs() + TINY[BF16], "drows")
            terms = dy[t].double() * rows[r].double()
            close(dw[t, k], terms.sum(), (H + 8) * 2.0 ** -24 * terms.abs().sum(), "dtopk_w")
        close(out[t], exact, 2.0 ** -8 * exact.abs() + 2.0 ** -21 * size + TINY[BF16], "combine")


def test_route_infinite_logits(mx):
    """+inf is chosen first; a softmax over it has no value, sigmoids have one."""
    logits = torch.tensor([[0.0, INF, -1.0, 2.0]], device="cuda")
    ids, w = mx.route_topk(logits, 2)
    assert ids.tolist() == [[1, 3]] and w.isnan().all()
    ids, w = mx.route_topk(logits, 2, score="sigmoid")
    assert ids.tolist() == [[1, 3]] and w[0, 0] == 1
    ids, w = mx.route_topk(logits, 3, bias=torch.tensor([0.0, -INF, 5.0, NAN], device="cuda"), score="sigmoid")
    assert ids.tolist() == [[2, 0, -1]] and w[0, 2] == 0
