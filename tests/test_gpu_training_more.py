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
