"""Tensors on several GPUs, on the CPU: stand-ins say which GPU they are on,
the library is one that records its calls. Nothing may reach it unless every
tensor, and a stream given, is on the current GPU."""
import pytest
import torch

from expanded_layout_expert_gb300 import Layout, training


class On(torch.Tensor):
    """A CPU tensor that says it is on GPU `gpu`."""

    @classmethod
    def __torch_function__(cls, func, types, args=(), kwargs=None):
        t = next((a for a in args if isinstance(a, On)), None)
        name = getattr(func, "__name__", "")
        if func is torch.Tensor.get_device:
            return t.gpu
        if func == torch.Tensor.is_cuda.__get__:
            return t.gpu >= 0
        if func == torch.Tensor.device.__get__:
            return torch.device("cuda", t.gpu) if t.gpu >= 0 else torch.device("cpu")
        out = super().__torch_function__(func, types, args, kwargs or {})
        if isinstance(out, On) and name != "__set__":
            out.gpu = t.gpu
        return out


def on(gpu, *shape, dtype=torch.float32):
    t = torch.ones(*shape).to(dtype).as_subclass(On)
    t.gpu = gpu
    return t


class Stream:
    cuda_stream = 0

    def __init__(self, gpu):
        self.device_index = gpu


@pytest.fixture
def calls(monkeypatch):
    got = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: got.append(name) or 0

    monkeypatch.setattr(training, "load", Library)
    monkeypatch.setattr(training, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    return got


BF16, I32 = torch.bfloat16, torch.int32


def layout(gpu, E=2, M=8):
    i32 = lambda *s: on(gpu, *s, dtype=I32)  # noqa: E731
    return Layout(psum=i32(E), start=i32(E), total=i32(1), m_indices=i32(M), src2dst=i32(4, 2),
                  tile_prefix=i32(E + 1), E=E, align=1, M_cap=M)


def arguments():
    """name -> (function, its tensors by name with their shapes and types)"""
    return {
        "expand_rows": (training.expand_rows, dict(
            x=(4, 16, BF16), topk_w=(4, 2, torch.float32), n_valid=(1, I32), out=(8, 16, BF16),
            row_w=(8, torch.float32), status=(1, I32))),
        "collect_row_grads": (training.collect_row_grads, dict(
            rows=(8, torch.float32), n_valid=(1, I32), out=(4, 2, torch.float32))),
        "grouped_matmul": (training.grouped_matmul, dict(
            x=(8, 16, BF16), w=(2, 24, 16, BF16), out=(8, 24, BF16), status=(1, I32))),
        "grouped_matmul_dgrad": (training.grouped_matmul_dgrad, dict(
            dy=(8, 24, BF16), w=(2, 24, 16, BF16), out=(8, 16, BF16), status=(1, I32))),
        "grouped_matmul_wgrad": (training.grouped_matmul_wgrad, dict(
            dy=(8, 24, BF16), x=(8, 16, BF16), out=(2, 24, 16, torch.float32), status=(1, I32))),
        "swiglu": (training.swiglu, dict(gu=(8, 32, BF16), row_w=(8, torch.float32), out=(8, 16, BF16))),
        "swiglu_backward": (training.swiglu_backward, dict(
            dh=(8, 16, BF16), gu=(8, 32, BF16), row_w=(8, torch.float32), dgu=(8, 32, BF16),
            drow_w=(8, torch.float32))),
    }


@pytest.mark.parametrize("name", arguments())
def test_calls(calls, name):
    f, shapes = arguments()[name]

    def call(lay=0, stream=None, **where):
        return f(**{k: on(where.get(k, where.get("all", 0)), *s[:-1], dtype=s[-1]) for k, s in shapes.items()},
                 lay=layout(lay), stream=stream)

    call()
    call(stream=Stream(0))
    assert len(calls) == 2
    for k in shapes:   # one tensor elsewhere: on another GPU, on the host
        for gpu in (1, -1):
            with pytest.raises(ValueError):
                call(**{k: gpu})
    for kw in (dict(lay=1), dict(all=1, lay=1), dict(all=1, lay=1, stream=Stream(1)), dict(stream=Stream(1))):
        with pytest.raises(ValueError):
            call(**kw)
    assert len(calls) == 2


def optimizer(gpus=(0, 0)):
    states = lambda: [on(g, 4) for g in gpus]  # noqa: E731
    return training.AdamW([on(g, 4) for g in gpus], exp_avg=states(), exp_avg_sq=states())


def test_adamw(calls, monkeypatch):
    with pytest.raises(ValueError, match="an optimizer for each GPU"):
        optimizer((0, 1))
    opt = optimizer()
    opt.step([on(0, 4), on(0, 4)], grad_scale=on(0, 1))
    opt.step([on(0, 4), on(0, 4)], stream=Stream(0))
    for grads, kw in (([on(0, 4), on(1, 4)], {}), ([on(0, 4), on(0, 4)], dict(grad_scale=on(1, 1))),
                      ([on(0, 4), on(0, 4)], dict(stream=Stream(1)))):
        with pytest.raises(ValueError):
            opt.step(grads, **kw)
    monkeypatch.setattr(training, "_current_device", lambda: 1, raising=False)
    with pytest.raises(ValueError):   # the launch would go to the other GPU
        opt.step([on(0, 4), on(0, 4)])
    assert calls == ["moe_adamw_step"] * 2 and opt.steps == 2


def test_layer_of_two_devices():
    with pytest.raises(ValueError, match="same GPU"):
        training.TrainableExperts(on(0, 2, 32, 16, dtype=BF16), on(1, 2, 16, 16, dtype=BF16), K=1, max_tokens=4)
