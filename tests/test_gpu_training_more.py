"""The training operators on the GPU, further cases: streams, capture, long
runs of the optimizer, refusals that must leave a layer as it was, products
that take the less travelled ways through the kernels."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F16, F32, F64 = torch.bfloat16, torch.float16, torch.float32, torch.float64


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


def layout_of(mx, counts):
    """A Layout with the given rows per expert, one pair per row."""
    counts = torch.tensor(counts, dtype=torch.int64)
    end = counts.cumsum(0)
    M = max(1, int(end[-1]))
    i32 = lambda t: t.to(torch.int32).cuda()  # noqa: E731
    return mx.Layout(psum=i32(end), start=i32(end - counts), total=i32(end[-1:]),
                     m_indices=i32(torch.empty(0)), src2dst=i32(torch.zeros(M, 1)),
                     tile_prefix=i32(torch.empty(0)), E=len(counts), align=1, M_cap=M), \
        list(zip((end - counts).tolist(), end.tolist()))


def test_results_are_made_on_the_calls_stream(mx):
    """The current stream is busy for longer than the call on another stream
    takes: what the call makes itself may neither wait for it nor be zeroed or
    given away by it."""
    lay, _ = layout_of(mx, [130, 7])
    g = gen(5)
    w, x = normal(g, 2, 256, 128, dtype=BF16), normal(g, lay.M_cap, 128, dtype=BF16)
    dy, gu = normal(g, lay.M_cap, 256, dtype=BF16), normal(g, lay.M_cap, 64, dtype=BF16)
    calls = [lambda s: mx.grouped_matmul(x, w, lay, stream=s), lambda s: mx.grouped_matmul_dgrad(dy, w, lay, stream=s),
             lambda s: mx.grouped_matmul_wgrad(dy, x, lay, stream=s), lambda s: mx.swiglu(gu, lay, stream=s),
             lambda s: mx.swiglu_backward(gu[:, :32], gu, lay, stream=s)[0],
             lambda s: mx.swiglu_backward(gu[:, :32], gu, lay, stream=s)[1]]
    want = [f(None) for f in calls]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(400_000_000)   # about 0.2 s
    got = [f(side) for f in calls]
    side.synchronize()
    with torch.cuda.stream(side):
        early = [t.clone() for t in got]
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(early, want))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_is_not_captured(mx, bits):
    """A graph would repeat one step's bias correction: the capture is refused,
    and the optimizer is as it was."""
    p, g = torch.ones(300, device="cuda"), torch.ones(300, device="cuda")
    q = p.clone()
    a, b = (mx.AdamW([t], state_bits=bits) for t in (p, q))
    a.step([g])
    b.step([g])
    torch.cuda.synchronize()
    with pytest.raises(mx.MoEError, match="captur"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            a.step([g])
    torch.cuda.synchronize()
    assert a.steps == 1 and torch.equal(p, q)
    a.step([g])
    b.step([g])
    assert a.steps == 2 and torch.equal(p, q)


def test_training_loop_around_a_graph(mx):
    """Forward and backward replayed from a graph, the optimizer's step between
    the replays, against the same loop without a graph."""
    T, K, E, H, I = 48, 2, 4, 128, 64

    def loop(graphed):
        g = gen(3)
        masters = [normal(g, E, 2 * I, H, std=0.1), normal(g, E, H, I, std=0.1)]
        layer = mx.TrainableExperts(*(t.bfloat16() for t in masters), K=K, max_tokens=T)
        opt = mx.AdamW(masters, copies=layer.parameters, lr=1e-2)
        x, dy = normal(g, T, H, dtype=BF16), normal(g, T, H, dtype=BF16)
        w, ids = torch.rand(T, E, generator=g, device="cuda").topk(K, dim=1)
        ids, w = ids.to(torch.int32).contiguous(), w.contiguous()
        layer.forward(x, ids, w)
        layer.backward(dy)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        if graphed:
            with torch.cuda.graph(graph):
                layer.forward(x, ids, w)
                layer.backward(dy)
        for _ in range(4):
            if graphed:
                graph.replay()
            else:
                layer.forward(x, ids, w)
                layer.backward(dy)
            opt.step(layer.gradients)
        torch.cuda.synchronize()
        return masters + layer.parameters

    assert all(torch.equal(a, b) for a, b in zip(loop(True), loop(False)))


# ------------------------------------------- AdamW with 8-bit states, long runs
def decoded(codes, scales):
    return codes.view(torch.float8_e4m3fn).float() * scales.repeat_interleave(128)[: codes.numel()]


@pytest.mark.parametrize("b2,small,steps", [(0.97, 0.01, 2000), (0.98, 0.01, 2000), (0.99, 0.01, 3000),
                                            (0.999, 0.3, 4000)])
def test_adamw_8_bit_states_follow_their_gradients(mx, b2, small, steps):
    """Half of every block's gradients fall to a fraction; the stored root
    against that of 32-bit states over the same gradients.

    A step's rounding moves a root by about its own change and its block's
    scale's, (1 - b2) together, times the step of a code (6-12 %, 9 on average)
    in variance, and the average forgets at 1 - b2, so its logarithm has a
    variance of 0.045; a fall by a factor D on the way adds log(D) * 0.09 (a
    walk of code steps), at most 0.11 for D = 3.3 (the others' fall is
    forgotten). One deviation is up to 0.4, 1 % and 99 % are at 2.33 of them:
    factors of 0.39 and 2.54; the median is within exp(-var / 2) = 0.93, taken
    twice as wide."""
    n = 12800
    g = gen(1)
    p, q = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    eight = mx.AdamW([p], state_bits=8, betas=(0.9, b2), lr=1e-3, weight_decay=0.0)
    full = mx.AdamW([q], betas=(0.9, b2), lr=1e-3, weight_decay=0.0)
    scale = torch.ones(n, device="cuda")
    moved = []
    for t in range(steps):
        if t == steps // 4:
            scale[::2] = small
        grad = torch.randn(n, generator=g, device="cuda") * scale
        before = p.clone(), q.clone()
        eight.step([grad])
        full.step([grad])
        if t >= steps - 50:
            moved.append([float((a - b)[::2].square().mean()) for a, b in zip((p, q), before)])
    ratio = decoded(eight.exp_avg_sq[0], eight.exp_avg_sq_scale[0]) / full.exp_avg_sq[0].sqrt()
    for half in (ratio[::2], ratio[1::2]):
        low, mid, high = torch.quantile(half, torch.tensor([0.01, 0.5, 0.99], device="cuda")).tolist()
        assert 0.86 < mid < 1.16 and low > 0.39 and high < 2.54, (low, mid, high)
    # and the steps are as large: m / r, with r's deviation of up to 0.4
    a, b = torch.tensor(moved).mean(0).sqrt().tolist()
    assert 0.7 < a / b < 1.5, (a, b)


def test_adamw_random_rounding_has_an_exact_mean(mx):
    """Every code, 25400 times, through one step without gradients beside a
    largest value that stays: each comes out as one of its value's two
    neighbours, on average as the value itself; the same again, and otherwise
    at another step or place in the list."""
    b1, b2, t = 0.9, 0.999, 5000
    start = torch.full((126, 200, 128), 126, dtype=torch.uint8, device="cuda")   # a block's first value: its largest
    start[:, :, 1:] = torch.arange(1, 127, dtype=torch.uint8, device="cuda")[:, None, None]
    grad = torch.zeros(126, 200, 128, device="cuda")
    grad[:, :, 0] = 448.0
    start, grad = start.reshape(-1), grad.reshape(-1)
    n = start.numel()
    sign = torch.where(torch.arange(n, device="cuda") % 2 == 0, 0, 128).to(torch.uint8)

    def run(step, place=0):
        zeros = lambda dtype=F32, count=8: [torch.zeros(count, dtype=dtype, device="cuda")] * place  # noqa: E731
        one = torch.ones(n // 128, device="cuda")
        opt = mx.AdamW(zeros() + [torch.zeros(n, device="cuda")], state_bits=8, betas=(b1, b2),
                       weight_decay=0.0, step=step, exp_avg=zeros(torch.uint8) + [start | sign],
                       exp_avg_sq=zeros(torch.uint8) + [start.clone()],
                       exp_avg_scale=zeros(F32, 1) + [one], exp_avg_sq_scale=zeros(F32, 1) + [one.clone()])
        opt.step(zeros() + [grad])
        return opt.exp_avg[-1], opt.exp_avg_scale[-1], opt.exp_avg_sq[-1], opt.exp_avg_sq_scale[-1]

    m, ms, v, vs = run(t)
    again, other, moved = run(t), run(t + 1), run(t, place=1)
    assert torch.equal(m, again[0]) and torch.equal(v, again[2])
    assert not torch.equal(m, other[0]) and not torch.equal(v, other[2])
    assert not torch.equal(v, moved[2])
    table = torch.arange(0, 127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).float()
    was = start.view(torch.float8_e4m3fn).float()
    for got, scale, factor, signed in ((m, ms, b1, True), (v, vs, b2 ** 0.5, False)):
        value = (got & 127).view(torch.float8_e4m3fn).float()
        if signed:
            assert torch.equal((got & 128)[value > 0], sign[value > 0])
        exact = was.double() * factor / scale.repeat_interleave(128).double()   # in the block's new scale
        exact[grad > 0] = 448.0
        low = torch.searchsorted(table.double(), exact * (1 - 2.0 ** -20), right=True) - 1
        high = torch.searchsorted(table.double(), exact * (1 + 2.0 ** -20)).clamp(max=126)
        at = (got & 127).long()
        assert ((at >= low) & (at <= high)).all()
        inner = torch.ones_like(got, dtype=torch.bool).view(-1, 128)
        inner[:, 0] = False
        for c in range(1, 127):
            these = (start == c) & inner.view(-1)
            if not signed and c == 1:
                assert (at[these] == 1).all()    # a positive root never becomes zero
                continue
            x, mean = value[these].double(), float(exact[these].mean())
            below, above = table[table <= mean].max().item(), table[table > mean].min().item()
            chance = (mean - below) / (above - below)
            # five deviations of a mean of len(x) roundings, one of them, and fp32's own
            sd = (above - below) * (chance * (1 - chance) / len(x)) ** 0.5
            assert abs(float(x.mean()) - mean) <= 5 * sd + (above - below) / len(x) + 2.0 ** -20 * mean, (c, factor)


@pytest.mark.parametrize("b1,b2", [(0.9, 0.95), (0.95, 0.95), (0.9, 0.98)])
def test_adamw_8_bit_states_of_values_without_gradients(mx, b1, b2):
    """Half of every block gets no gradients any more, while the other half
    does: its first moments reach zero and it stops moving. A first moment of
    the largest code is under the smallest after log(448 * 512) / -log(b1) =
    241 steps at 0.95; rounded at random (b2 = 0.98) it is then gone by each
    step with a chance of 1 - b1, and 450 more leave none."""
    n = 12800
    g = gen(2)
    p = torch.zeros(n, device="cuda")
    opt = mx.AdamW([p], state_bits=8, betas=(b1, b2), lr=1e-3, weight_decay=0.0)
    for t in range(1000):
        grad = normal(g, n)
        if t >= 200:
            grad[::2] = 0
        opt.step([grad])
        if t == 900:
            at = p.clone()
    assert (opt.exp_avg[0][::2] & 127 == 0).all()
    assert torch.equal(p[::2], at[::2]) and not torch.equal(p[1::2], at[1::2])


def test_adamw_8_bit_states_of_blocks_without_gradients(mx):
    """No gradient in a whole block (an expert without tokens): the moments
    decay with the block's scale, as they do in 32 bits, and the codes stay,
    but for m's below 2^-6, which become zero."""
    n = 12800
    g = gen(4)
    p, q, grad = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda"), normal(g, n)
    eight = mx.AdamW([p], state_bits=8, betas=(0.9, 0.95), weight_decay=0.0)
    full = mx.AdamW([q], betas=(0.9, 0.95), weight_decay=0.0)
    for opt in (eight, full):
        opt.step([grad])
    codes = eight.exp_avg[0].clone(), eight.exp_avg_sq[0].clone()
    for _ in range(40):
        for opt in (eight, full):
            opt.step([torch.zeros_like(grad)])
    assert torch.equal(eight.exp_avg_sq[0], codes[1])
    assert torch.equal(eight.exp_avg[0] & 127, torch.where(codes[0] & 127 < 8, 0, codes[0] & 127))
    for scales, value in ((eight.exp_avg_scale[0], full.exp_avg[0]), (eight.exp_avg_sq_scale[0], full.exp_avg_sq[0].sqrt())):
        want = value.abs().view(-1, 128).amax(1) / 448
        assert ((scales - want).abs() <= 50 * 2.0 ** -22 * want).all()


@pytest.mark.parametrize("name,dtype,count", [("exp_avg", torch.uint8, 256), ("exp_avg_scale", F32, 2),
                                              ("exp_avg_sq", torch.uint8, 256), ("exp_avg_sq_scale", F32, 2)])
def test_adamw_checkpoint_in_part_is_refused(mx, name, dtype, count):
    """8-bit codes without their scales (or scales without codes) would go on
    as zeros."""
    p = torch.zeros(256, device="cuda")
    with pytest.raises(ValueError, match="come together"):
        mx.AdamW([p], state_bits=8, **{name: [torch.ones(count, dtype=dtype, device="cuda")]})


# --------------------------------------------------------------- the layer
def small_layer(mx, T=16, K=2, E=4, H=64, I=64):
    g = gen(1)
    layer = mx.TrainableExperts(normal(g, E, 2 * I, H, dtype=BF16, std=0.1), normal(g, E, H, I, dtype=BF16, std=0.1),
                                K=K, max_tokens=T)
    w, ids = torch.rand(T, E, generator=g, device="cuda").topk(K, dim=1)
    return layer, normal(g, T, H, dtype=BF16), ids.to(torch.int32).contiguous(), w.contiguous()


def test_refused_calls_leave_the_forward(mx):
    """A forward or backward refused for its arguments leaves the forward
    before it, and the backward that belongs to it, as they were."""
    layer, x, ids, w = small_layer(mx)
    layer.forward(x, ids, w)
    layer.backward(x)
    want = [t.clone() for t in (layer.dx, layer.dtopk_w, *layer.gradients)]
    layer.forward(x, ids, w)
    other = ids.flip(0).contiguous()
    for bad in ((x.float(), other, w), (x, other.long(), w), (x, other, w.double()), (x, other, None),
                (x, other, w, torch.ones(1, device="cuda")), (x, other, w[:, :1])):
        with pytest.raises(ValueError):
            layer.forward(*bad)
    for bad in (x.float(), x.half(), x[:-1], x[:, :-8]):
        with pytest.raises(ValueError):
            layer.backward(bad)
    with pytest.raises(mx.MoEError):   # rows that do not begin on 16 bytes
        layer.backward(torch.zeros(16, 72, dtype=BF16, device="cuda")[:, 1:65])
    layer.backward(x)
    assert all(torch.equal(a, b) for a, b in zip(want, (layer.dx, layer.dtopk_w, *layer.gradients)))
    # refused by the library, once the layout was made: no backward of a mixture
    layer.forward(x, ids, w)
    with pytest.raises(mx.MoEError):
        layer.forward(torch.zeros(16, 72, dtype=BF16, device="cuda")[:, 1:65], other, w)
    with pytest.raises(RuntimeError):
        layer.backward(x)


@pytest.mark.parametrize("side", [False, True])
def test_n_valid_belongs_to_the_forward(mx, side):
    """A caller may refill its word (and x) for the next batch before the
    backward, which takes the forward's."""
    layer, x, ids, w = small_layer(mx)
    n_valid = torch.tensor([9, 5], dtype=torch.int32, device="cuda")
    stream = torch.cuda.Stream() if side else None
    torch.cuda.synchronize()
    results = []
    for refill in (False, True):
        mine, word = x.clone(), n_valid.clone()
        torch.cuda.synchronize()
        layer.forward(mine, ids, w, word, stream=stream)
        torch.cuda.synchronize()
        if refill:
            word.fill_(14)
            mine.fill_(float("nan"))
            torch.cuda.synchronize()
        layer.dx.fill_(7)
        layer.dtopk_w.fill_(7)
        torch.cuda.synchronize()
        layer.backward(x, stream=stream)
        torch.cuda.synchronize()
        results.append([t.clone() for t in (layer.dx, layer.dtopk_w, *layer.gradients)])
        assert (layer.dx[9:] == 7).all() and (layer.dtopk_w[9:] == 7).all() and not (layer.dx[:9] == 7).any()
    assert all(torch.equal(a, b) for a, b in zip(*results))


def test_n_valid_in_a_graph(mx):
    """The word is copied by the graph, at each replay."""
    layer, x, ids, w = small_layer(mx)
    n_valid = torch.tensor([16], dtype=torch.int32, device="cuda")

    def once():
        layer.forward(x, ids, w, n_valid)
        layer.backward(x)

    once()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        once()
    for n in (16, 3, 11):
        n_valid.fill_(n)
        once()
        want = [t.clone() for t in (layer.dx[:n], *layer.gradients)]
        layer.dx.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, (layer.dx[:n], *layer.gradients)))
        assert (layer.dx[n:] == 0).all()


# --------------------------------------------------------------- the products
U = {BF16: 2.0 ** -8, F16: 2.0 ** -11, F32: 2.0 ** -24}


def near(got, a, b, dtype, what):
    """got = a b^T rounded to dtype, a [i, c] and b [j, c] in 64 bits, by the
    norm: each result is off by half a step at most, and each of its sum's c / 16
    additions of 16 products by a step of fp32 at most (the tensor core
    truncates). A lost term of 4104 is 1.6 % of the norm, the bound 0.5 %."""
    exact = a @ b.T
    bound = U[dtype] * float(exact.norm()) + (a.shape[1] // 16 + 1) * 2.0 ** -23 * float((a.abs() @ b.abs().T).norm())
    assert float((got.double() - exact).norm()) <= bound, what


def operands(mx, counts, N, Kd, dtype, seed=0):
    lay, bounds = layout_of(mx, counts)
    g = gen(seed + N + Kd)
    x, dy = normal(g, lay.M_cap, Kd, dtype=dtype), normal(g, lay.M_cap, N, dtype=dtype)
    return lay, bounds, x, dy, normal(g, lay.E, N, Kd, dtype=dtype, std=0.1)


def check_products(mx, lay, bounds, x, dy, w, only=None):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = mx.grouped_matmul(x, w, lay, status=status)
    dx = mx.grouped_matmul_dgrad(dy, w, lay, status=status)
    dw = {t: mx.grouped_matmul_wgrad(dy, x, lay, out_dtype=t, status=status) for t in (x.dtype, F32)}
    assert status.item() == 0
    for e, (a, b) in enumerate(bounds):
        if only is not None and e not in only:
            continue
        if a == b:
            assert all((t[e] == 0).all() for t in dw.values())
            continue
        X, DY, W = x[a:b].double(), dy[a:b].double(), w[e].double()
        near(y[a:b], X, W, x.dtype, f"forward {e}")
        near(dx[a:b], DY, W.T, x.dtype, f"dgrad {e}")
        for t, got in dw.items():
            near(got[e], DY.T, X.T, t, f"wgrad {t} {e}")


@pytest.mark.parametrize("E,N,Kd", [(33, 136, 520), (160, 264, 72), (160, 40, 264), (1024, 40, 64)])
def test_many_experts_with_many_rows(mx, E, N, Kd):
    """Over 40 rows an expert on average, so the pairs take them: several
    experts a thread and several warps in the search for a tile's expert."""
    counts = [0 if e % 11 == 5 else (e * 37) % 131 + (300 if e % 40 == 7 else 0) for e in range(E)]
    assert sum(counts) > 40 * E
    only = None if E <= 160 else set(range(0, E, 13)) | {E - 1}
    check_products(mx, *operands(mx, counts, N, Kd, BF16), only=only)


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("counts", [[4700, 3, 2049], [1, 2048, 2047, 0, 5000]], ids=["a", "b"])
def test_experts_with_many_row_tiles(mx, counts, dtype):
    """More than eight tiles of 256 rows, several columns of tiles: the order of
    the tiles begins a second column of its own."""
    check_products(mx, *operands(mx, counts, 1032, 776, dtype))


@pytest.mark.parametrize("counts", [[1400] + [(e * 7) % 61 for e in range(159)], [0] * 63 + [2500]],
                         ids=["skewed", "one of 64"])
def test_few_rows_on_average(mx, counts):
    """At most 40 rows an expert on average, most of them with one expert."""
    assert sum(counts) <= 40 * len(counts)
    check_products(mx, *operands(mx, counts, 520, 1032, BF16), only={0, 1, 2, 30, len(counts) - 1})


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("N,Kd", [(136, 4104), (4104, 136), (2048, 768)])
def test_long_contractions(mx, N, Kd, dtype):
    """No term of a long sum is lost, whole and split over a cluster, few rows
    and many."""
    check_products(mx, *operands(mx, [1, 9, 0, 30, 5], N, Kd, dtype))
    check_products(mx, *operands(mx, [700, 64, 0, 351], N, Kd, dtype))


@pytest.mark.parametrize("mean", [0.0, 0.5])
def test_long_sums_of_many_tiles_do_not_drift(mx, mean):
    """wgrad with too many tiles to share an expert's rows among CTAs: pairs,
    whose sums leave the tensor core after at most 56 additions (896 rows),
    each truncated by 2^-24 of its size at most, as in the shared form."""
    lay, bounds = layout_of(mx, [16384, 0, 897])
    g = gen(6)
    x = (normal(g, lay.M_cap, 1032) + mean).to(BF16)
    dy = (normal(g, lay.M_cap, 1032) + mean).to(BF16)
    base = normal(g, 3, 1032, 1032)
    dw = mx.grouped_matmul_wgrad(dy, x, lay, out_dtype=F32)
    added = mx.grouped_matmul_wgrad(dy, x, lay, out=base.clone(), accumulate=True)
    for e, (a, b) in enumerate(bounds):
        r = dy[a:b].double().T @ x[a:b].double()
        for got, want in ((dw[e], r), (added[e], r + base[e].double())):
            assert float((got.double() - want).norm()) <= 60 * 2.0 ** -24 * float(want.norm())


# ------------------------------------------------------ gradients not finite
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("bits,b2", [(32, 0.95), (8, 0.95), (8, 0.999)])
def test_adamw_gradients_that_are_not_finite(mx, bits, b2, value):
    """Each spoils its own parameter at once; with 8-bit states the rest of
    its block of 128 is right at this step and the other blocks always."""
    n, at = 1000, [5, 300, 301, 302, 303, 999]
    g = gen(8)
    start, grads = normal(g, n), [normal(g, n) for _ in range(30)]
    p, q, copy = start.clone(), start.clone(), torch.zeros(n, dtype=BF16, device="cuda")
    bad = mx.AdamW([p], copies=[copy], state_bits=bits, betas=(0.9, b2))
    good = mx.AdamW([q], state_bits=bits, betas=(0.9, b2))
    spoilt = torch.zeros(n, dtype=torch.bool, device="cuda")
    spoilt[at] = True
    for t in range(26):
        bad.step([grads[t]])
        good.step([grads[t]])
    wrong = grads[26].clone()
    wrong[at] = value
    bad.step([wrong])
    good.step([grads[26]])
    assert p[spoilt].isnan().all() and torch.equal(p[~spoilt], q[~spoilt])
    assert torch.equal(copy[~spoilt], q[~spoilt].bfloat16()) and copy[spoilt].isnan().all()
    if bits == 8:
        spoilt = spoilt.nonzero().view(-1) // 128
        spoilt = torch.isin(torch.arange(n, device="cuda") // 128, spoilt)
    for t in range(27, 30):
        bad.step([grads[t]])
        good.step([grads[t]])
    assert torch.equal(p[~spoilt], q[~spoilt]) and p[at].isnan().all()
    for a, b in zip((bad.exp_avg[0], bad.exp_avg_sq[0]), (good.exp_avg[0], good.exp_avg_sq[0])):
        assert torch.equal(a[~spoilt], b[~spoilt])


def test_expand_rows_of_segments_outside_the_buffer(mx):
    """Ends before the buffer or past it: only rows inside are zeroed (the
    buffer is the middle of a larger one)."""
    lay, _ = layout_of(mx, [5, 5, 5, 5])
    lay.align, lay.src2dst = 16, torch.full((4, 2), -1, dtype=torch.int32, device="cuda")
    lay.psum = torch.tensor([-7, 20, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
    large = torch.full((60, 64), 5.0, dtype=BF16, device="cuda")
    weights = torch.full((60,), 5.0, device="cuda")
    mx.expand_rows(torch.ones(4, 64, dtype=BF16, device="cuda"), lay, torch.ones(4, 2, device="cuda"),
                   out=large[20:40], row_w=weights[20:40])
    assert (large[:20] == 5).all() and (large[40:] == 5).all()
    assert (weights[:20] == 5).all() and (weights[40:] == 5).all()
    assert (large[20:40] == 5).all() and (weights[20:40] == 5).all()   # 0 and 20 end on no gap inside


@pytest.mark.parametrize("rows,N", [(896, 136), (16384, 136), (16384, 1032)], ids=["short", "shared", "pairs"])
@pytest.mark.parametrize("mean", [0.0, 0.5])
def test_fp32_sums_of_rows(mx, rows, N, mean):
    """wgrad into fp32, by the norm. The tensor core adds 16 rows at a time
    and truncates: half a step, 0.72 * 2^-24 of the sum so far, which is half of
    the whole on average. At most 32 additions (512 rows) follow one another,
    then the partial sums are rounded to nearest: 32 / 2 * 0.72 * 2^-24."""
    lay, bounds = layout_of(mx, [rows, rows])
    g = gen(3)
    x = (normal(g, lay.M_cap, 1032) + mean).to(BF16)
    dy = (normal(g, lay.M_cap, N) + mean).to(BF16)
    dw = mx.grouped_matmul_wgrad(dy, x, lay, out_dtype=F32)
    for e, (a, b) in enumerate(bounds):
        r = dy[a:b].double().T @ x[a:b].double()
        assert float((dw[e].double() - r).norm()) <= 11.5 * 2.0 ** -24 * float(r.norm())


def test_adamw_random_rounding_of_many_tensors(mx):
    """Every tensor of the list has bits of its own, those of a second launch
    (from the 401st on) too; empty ones have no place."""
    n, count = 512, 802
    start, grad = torch.full((n,), 100, dtype=torch.uint8, device="cuda"), torch.zeros(n, device="cuda")
    start[::128], grad[::128] = 126, 448.0
    none = torch.zeros(0, device="cuda")

    def run(empty):
        params = [torch.zeros(n, device="cuda") for _ in range(count)]
        codes = lambda: [start.clone() for _ in range(count)]  # noqa: E731
        ones = lambda: [torch.ones(n // 128, device="cuda") for _ in range(count)]  # noqa: E731
        pad = [none] * empty
        opt = mx.AdamW(pad + params, state_bits=8, betas=(0.9, 0.999), weight_decay=0.0, step=5000,
                       exp_avg=[none.byte()] * empty + codes(), exp_avg_sq=[none.byte()] * empty + codes(),
                       exp_avg_scale=pad + ones(), exp_avg_sq_scale=pad + ones())
        opt.step(pad + [grad] * count)
        return torch.stack(opt.exp_avg[empty:])

    m = run(0)
    assert len(torch.unique(m, dim=0)) == count
    assert torch.equal(m, run(3))
