"""The operators of routing.py and w4.py together, as the layers use them:
TrainableExperts with weights applied in the return, from the router's logits to
their gradient; FourBitExperts for decode batches, captured and replayed."""
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


def near(got, want, limit, what):
    fro = float((got.double() - want).norm() / want.norm().clamp(min=1e-300))
    assert fro <= limit, (what, fro)


@pytest.mark.parametrize("score,renormalize", [("softmax", False), ("softmax", True), ("sigmoid", True)])
@pytest.mark.parametrize("T,K,E,H,I,align,nv", [(37, 2, 6, 128, 64, 1, 30), (300, 4, 8, 256, 136, 16, 300),
                                                (1, 1, 3, 64, 64, 128, 1)])
def test_training_from_the_logits(mx, T, K, E, H, I, align, nv, score, renormalize):
    """Router, experts and weighted return, forward and back, against autograd of
    the formula in 64 bits on the same bf16 inputs. Every intermediate is rounded
    to bf16 once (2^-8 at most), four roundings deep: 2 % of the result's norm."""
    g = gen(T)
    w13 = normal(g, E, 2 * I, H, dtype=BF16, std=H ** -0.5)
    w2 = normal(g, E, H, I, dtype=BF16, std=I ** -0.5)
    x, dy = normal(g, T, H, dtype=BF16), normal(g, T, H, dtype=BF16)
    logits = normal(g, T, E)
    if T > 10:
        logits[4, 1:] = -float("inf")   # one expert left
        logits[6] = -float("inf")       # none: an inactive token
    n_valid = torch.tensor([nv], dtype=torch.int32, device="cuda")
    layer = mx.TrainableExperts(w13, w2, K=K, max_tokens=T, align=align, weighting="gather")
    ids, w = mx.route_topk(logits, K, score=score, renormalize=renormalize, factor=1.5, n_valid=n_valid)
    kept_w = w.clone()
    y = layer.forward(x, ids, w, n_valid).clone()
    w.fill_(float("nan"))   # the layer keeps its own copy for the backward
    dx, dw = (t.clone() for t in layer.backward(dy))
    grads = [t.clone() for t in layer.gradients]
    dl = mx.route_topk_backward(dw, logits, ids, score=score, renormalize=renormalize, factor=1.5, n_valid=n_valid)
    torch.cuda.synchronize()
    assert layer.status.item() == 0
    X, L = x[:nv].double().requires_grad_(), logits[:nv].double().requires_grad_()
    W13, W2 = w13.double().requires_grad_(), w2.double().requires_grad_()
    picked = torch.zeros(nv, E, dtype=torch.bool, device="cuda")
    for k in range(K):
        t = torch.nonzero(ids[:nv, k] >= 0)[:, 0]
        picked[t, ids[t, k].long()] = True
    dead = ~picked.any(1, keepdim=True)
    safe = torch.where(L.isfinite(), L, -1e30)
    if score == "softmax":
        p = torch.softmax(safe.masked_fill(~picked, -1e30) if renormalize else safe, 1)
    else:
        p = torch.sigmoid(safe) * picked
        p = p / torch.where(dead, 1.0, p.sum(1, keepdim=True))
    W = 1.5 * torch.where(picked, p, 0.0)
    out = torch.zeros(nv, H, dtype=F64, device="cuda")
    for e in range(E):
        t = torch.nonzero(picked[:, e])[:, 0]
        if len(t):
            G, V = (X[t] @ W13[e].T).split(I, dim=1)
            out = out.index_add(0, t, W[t, e][:, None] * ((torch.nn.functional.silu(G) * V) @ W2[e].T))
    out.backward(dy[:nv].double())
    near(y[:nv], out.detach(), 0.02, "y")
    near(dx[:nv], X.grad, 0.02, "dx")
    near(grads[0], W13.grad, 0.02, "dw13")
    near(grads[1], W2.grad, 0.02, "dw2")
    want = torch.nan_to_num(L.grad)
    if float(want.norm()) > 1e-12:
        # rounded rows make dtopk_w's errors; the softmax's gradient is a difference of them
        scale = (dw[:nv].double().norm() * 1.5)
        assert float((dl[:nv].double() - want).norm()) <= 0.02 * float(scale), "dlogits"
    assert (dl[nv:] == 0).all()
    # a second micro-batch adds to the weights' gradients
    layer.forward(x, ids, kept_w, n_valid)
    layer.backward(dy, accumulate=True)
    for a, b in zip(layer.gradients, grads):
        assert torch.equal(a, b + b)
    with pytest.raises(RuntimeError):
        layer.backward(dy)


def test_weightings_agree(mx):
    """The weight before the second product or after it: the same but for one
    rounding of the intermediate (2^-8) and one of the rows."""
    g = gen(3)
    T, K, E, H, I = 64, 3, 5, 192, 128
    w13, w2 = normal(g, E, 2 * I, H, dtype=BF16, std=H ** -0.5), normal(g, E, H, I, dtype=BF16, std=I ** -0.5)
    x, dy = normal(g, T, H, dtype=BF16), normal(g, T, H, dtype=BF16)
    ids, w = mx.route_topk(normal(g, T, E), K)
    a, b = (mx.TrainableExperts(w13, w2, K=K, max_tokens=T, weighting=how) for how in ("expanded", "gather"))
    near(b.forward(x, ids, w), a.forward(x, ids, w).double(), 0.01, "y")
    for u, v, what in zip(b.backward(dy), a.backward(dy), ("dx", "dtopk_w")):
        near(u, v.double(), 0.02, what)
    with pytest.raises(ValueError, match="weighting"):
        mx.TrainableExperts(w13, w2, K=K, max_tokens=T, weighting="rows")


def test_refused_calls_leave_the_forward_of_gather(mx):
    g = gen(4)
    T, K, E, H, I = 16, 2, 4, 64, 64
    layer = mx.TrainableExperts(normal(g, E, 2 * I, H, dtype=BF16), normal(g, E, H, I, dtype=BF16), K=K,
                                max_tokens=T, weighting="gather")
    x, dy = normal(g, T, H, dtype=BF16), normal(g, T, H, dtype=BF16)
    ids, w = mx.route_topk(normal(g, T, E), K)
    layer.forward(x, ids, w)
    want = [t.clone() for t in layer.backward(dy)]
    layer.forward(x, ids, w)
    for bad in (dy.float(), dy[:3], dy.half()):
        with pytest.raises(ValueError):
            layer.backward(bad)
    with pytest.raises(ValueError):
        layer.forward(x, ids, w.double())
    for a, b in zip(layer.backward(dy), want):
        assert torch.equal(a, b)


def test_training_of_gather_captured(mx):
    g = gen(5)
    T, K, E, H, I = 48, 2, 6, 128, 64
    layer = mx.TrainableExperts(normal(g, E, 2 * I, H, dtype=BF16, std=H ** -0.5),
                                normal(g, E, H, I, dtype=BF16, std=I ** -0.5), K=K, max_tokens=T,
                                weighting="gather")
    x, dy, logits = normal(g, T, H, dtype=BF16), normal(g, T, H, dtype=BF16), normal(g, T, E)

    def step():
        ids, w = mx.route_topk(logits, K, renormalize=True)
        y = layer.forward(x, ids, w)
        dx, dw = layer.backward(dy)
        return [y, dx, dw, mx.route_topk_backward(dw, logits, ids, renormalize=True), *layer.gradients]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in (1, 2):
        logits.copy_(normal(gen(seed), T, E))
        graph.replay()
        got = [t.clone() for t in held]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)


# ------------------------------------------------------------------ decode in 4 bits
def quantised(g, E, N, Kd, group, dtype, zeros, std):
    codes = torch.randint(0, 256, (E, N, Kd // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = ((torch.rand(E, N, Kd // group, generator=g, device="cuda") * 0.5 + 0.75) * std / 4.6).to(dtype)
    z = torch.randint(6, 10, (E, N, Kd // group), generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    return codes, scales, z


def dense(w):
    codes, scales, z = w
    q = torch.stack([codes & 15, codes >> 4], dim=3).flatten(2).double()
    group = q.shape[2] // scales.shape[2]
    off = 8.0 if z is None else z.double().repeat_interleave(group, 2)
    return (q - off) * scales.double().repeat_interleave(group, 2)


def four_bit_formula(x, ids, w, w13, w2, residual):
    I = w2.shape[2]
    out = torch.zeros(x.shape, dtype=F64, device="cuda") if residual is None else residual.double()
    for e in range(w13.shape[0]):
        t, k = torch.nonzero(ids == e, as_tuple=True)
        if len(t):
            G, V = (x[t].double() @ w13[e].T).split(I, dim=1)
            h = torch.nn.functional.silu(G) * V
            out = out.index_add(0, t, (h @ w2[e].T) * w[t, k].double()[:, None])
    return out


# three roundings of the intermediates and one of the result, each half a step at most
LIMIT = {BF16: 4 * 2.0 ** -8, F16: 4 * 2.0 ** -11}


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("T,K,E,H,I,group,zeros,align,nv", [
    (1, 4, 16, 512, 256, 128, True, 1, 1), (24, 2, 8, 256, 128, 32, False, 1, 20),
    (200, 4, 6, 384, 192, 64, True, 16, 200), (64, 8, 8, 1024, 512, 128, False, 1, 64)])
def test_four_bit_experts(mx, T, K, E, H, I, group, zeros, align, nv, dtype):
    g = gen(T + E)
    w13 = quantised(g, E, 2 * I, H, group, dtype, zeros, H ** -0.5)
    w2 = quantised(g, E, H, I, group, dtype, zeros, I ** -0.5)
    layer = mx.FourBitExperts(w13, w2, K=K, max_tokens=T, align=align)
    x, res = normal(g, T, H, dtype=dtype), normal(g, T, H, dtype=dtype)
    logits = normal(g, T, E)
    if T > 10:
        logits[3] = -float("inf")
    n_valid = torch.tensor([nv], dtype=torch.int32, device="cuda")
    ids, w = mx.route_topk(logits, K, renormalize=True, n_valid=n_valid)
    for residual in (None, res):
        y = layer.forward(x, ids, w, n_valid, residual=residual, out=torch.full_like(x, 7.0))
        assert layer.status.item() == 0
        want = four_bit_formula(x[:nv], ids[:nv], w[:nv], dense(w13), dense(w2),
                                None if residual is None else residual[:nv])
        near(y[:nv], want, LIMIT[dtype], "y")
        assert (y[nv:] == 7).all()
    # the residual's place may be the result's
    inplace = res.clone()
    assert layer.forward(x, ids, w, n_valid, residual=inplace, out=inplace) is inplace
    assert torch.equal(inplace[:nv], y[:nv]) and torch.equal(inplace[nv:], res[nv:])


def test_four_bit_experts_captured_and_on_another_stream(mx):
    """Two layers that share nothing, captured into two graphs and replayed in
    turn on new tokens; then a call queued behind a busy stream."""
    g = gen(11)
    T, K, E, H, I = 4, 4, 16, 512, 256
    layers = [mx.FourBitExperts(quantised(g, E, 2 * I, H, 128, BF16, True, H ** -0.5),
                                quantised(g, E, H, I, 128, BF16, True, I ** -0.5), K=K, max_tokens=T)
              for _ in range(2)]
    x, logits = normal(g, T, H, dtype=BF16), normal(g, T, E)

    def run(layer, out, stream=None):
        ids, w = mx.route_topk(logits, K, stream=stream)
        return layer.forward(x, ids, w, residual=x, out=out, stream=stream)

    outs = [torch.zeros(T, H, dtype=BF16, device="cuda") for _ in layers]
    graphs = []
    for layer, out in zip(layers, outs):
        run(layer, out)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run(layer, out)
        graphs.append(graph)
    for seed in (1, 2, 3):
        x.copy_(normal(gen(seed), T, H))
        logits.copy_(normal(gen(seed + 10), T, E))
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for layer, out in zip(layers, outs):
            assert torch.equal(out, run(layer, torch.empty_like(out)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    got = run(layers[0], torch.zeros_like(outs[0]), stream=side)
    side.synchronize()
    assert torch.equal(got, outs[0])


def test_four_bit_experts_refuse(mx):
    g = gen(12)
    w13, w2 = quantised(g, 4, 64, 128, 32, BF16, True, 0.1), quantised(g, 4, 128, 32, 32, BF16, True, 0.1)
    layer = mx.FourBitExperts(w13, w2, K=2, max_tokens=3)
    x, ids, w = normal(g, 3, 128, dtype=BF16), torch.zeros(3, 2, dtype=torch.int32, device="cuda"), \
        torch.ones(3, 2, device="cuda")
    layer.forward(x, ids, w)
    for bad in (dict(x=x.half()), dict(x=x[:2]), dict(topk_ids=ids.long()), dict(topk_w=w.double()),
                dict(topk_w=None), dict(residual=x.float()), dict(out=x.float())):
        with pytest.raises(ValueError):
            layer.forward(**{**dict(x=x, topk_ids=ids, topk_w=w), **bad})
    for bad in ((w13, w13), ((w13[0], w13[1].half(), w13[2]), w2), (w13, (w2[0][:3], w2[1][:3], w2[2][:3])),
                ((w13[0], w13[1], w13[2][:, :8]), w2), ((w13[0].cpu(), w13[1], w13[2]), w2)):
        with pytest.raises(ValueError):
            mx.FourBitExperts(*bad, K=2, max_tokens=3)


def test_four_bit_experts_overflow_is_flagged(mx):
    """An id past the last expert sets the status, and costs its pair alone."""
    g = gen(13)
    w13, w2 = quantised(g, 4, 64, 128, 32, F16, False, 0.1), quantised(g, 4, 128, 32, 32, F16, False, 0.1)
    layer = mx.FourBitExperts(w13, w2, K=2, max_tokens=3)
    x = normal(g, 3, 128, dtype=F16)
    ids = torch.tensor([[0, 1], [2, 9], [3, -1]], dtype=torch.int32, device="cuda")
    w = torch.ones(3, 2, device="cuda")
    y = layer.forward(x, ids, w).clone()
    assert layer.status.item() == -5
    ids[1, 1] = -1
    assert torch.equal(layer.forward(x, ids, w), y)
