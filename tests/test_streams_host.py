"""Results that a call makes itself are made on the stream that the call is
queued on, on the CPU: the library, the checks of the arguments and the stream
are stand-ins, and every tensor made is asked which stream was current."""
import contextlib

import pytest
import torch

import expanded_layout_expert_gb300 as mx
from expanded_layout_expert_gb300 import Layout, training


class Library:
    def __getattr__(self, name):
        return lambda *a: 0


@pytest.fixture
def made(monkeypatch):
    """[(stream current when a tensor was made)], with the calls' checks and
    the library replaced."""
    current, seen = [None], []

    @contextlib.contextmanager
    def stream(s):
        was, current[0] = current[0], s
        yield
        current[0] = was

    def recorded(make):
        def f(*a, **k):
            seen.append(current[0])
            return make(*a, **k)
        return f

    monkeypatch.setattr(torch.cuda, "stream", stream)
    for name in ("zeros", "empty"):
        monkeypatch.setattr(torch, name, recorded(getattr(torch, name)))
    monkeypatch.setattr(training, "load", Library)
    monkeypatch.setattr(training, "_rows", lambda t, *a: (0, t.shape[1]))
    for name in ("_whole", "_word", "_stream", "_device"):
        monkeypatch.setattr(training, name, lambda *a: 0, raising=False)
    monkeypatch.setattr(mx, "load", Library)
    monkeypatch.setattr(mx, "_stream", lambda *a: 0)
    monkeypatch.setattr(mx, "workspace_size", lambda *a: 16)
    return seen


def layout(E=2, M=8):
    i32 = lambda *s: torch.ones(*s, dtype=torch.int32)  # noqa: E731
    return Layout(psum=i32(E), start=i32(E), total=i32(1), m_indices=i32(M), src2dst=i32(4, 2),
                  tile_prefix=i32(E + 1), E=E, align=1, M_cap=M)


def bf16(*s):
    return torch.ones(*s).bfloat16()


CALLS = {
    "expand_rows": lambda s: training.expand_rows(bf16(4, 16), layout(), torch.ones(4, 2), stream=s),
    "collect_row_grads": lambda s: training.collect_row_grads(torch.ones(8), layout(), stream=s),
    "grouped_matmul": lambda s: training.grouped_matmul(bf16(8, 16), bf16(2, 24, 16), layout(), stream=s),
    "grouped_matmul_dgrad": lambda s: training.grouped_matmul_dgrad(bf16(8, 24), bf16(2, 24, 16), layout(),
                                                                    stream=s),
    "grouped_matmul_wgrad": lambda s: training.grouped_matmul_wgrad(bf16(8, 24), bf16(8, 16), layout(),
                                                                    stream=s),
    "swiglu": lambda s: training.swiglu(bf16(8, 32), layout(), stream=s),
    "swiglu_backward": lambda s: training.swiglu_backward(bf16(8, 16), bf16(8, 32), layout(), stream=s),
}


def u8(*s):
    return torch.ones(*s).to(torch.uint8)


IDS, SCALE = torch.ones(4, 2, dtype=torch.int32), torch.ones(4, 1)
CALLS.update({
    "expand_layout": lambda s: mx.expand_layout(IDS, 2, 1, 8, stream=s),
    "expand_scatter": lambda s: mx.expand_scatter(u8(4, 128), SCALE, 0, torch.ones(4, 2), layout(), stream=s),
    "expand_layout_scatter": lambda s: mx.expand_layout_scatter(u8(4, 128), SCALE, 0, IDS, torch.ones(4, 2), 2, 1,
                                                                8, stream=s),
    "grouped_gemm": lambda s: mx.grouped_gemm(u8(8, 128), torch.ones(8, 1), 0, layout(), u8(2, 128, 128), SCALE,
                                              stream=s),
    "act_quant": lambda s: mx.act_quant(bf16(8, 256), None, 0, 1, torch.ones(1), stream=s),
    "grouped_gemm_act_quant": lambda s: mx.grouped_gemm_act_quant(u8(8, 128), torch.ones(8, 1), 0, layout(),
                                                                  u8(2, 256, 128), SCALE, stream=s),
    "grouped_ffn": lambda s: mx.grouped_ffn(u8(8, 128), torch.ones(8, 1), 0, layout(), u8(2, 256, 128), SCALE,
                                            u8(2, 128, 128), SCALE, torch.ones(8), 0, stream=s),
})


@pytest.mark.parametrize("name", CALLS)
def test_results_are_made_on_the_calls_stream(made, name):
    side = object()
    CALLS[name](side)
    assert made and all(s is side for s in made)
    made.clear()
    CALLS[name](None)
    assert made and all(s is None for s in made)
