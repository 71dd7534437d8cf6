"""Refusals of the router, the weighted return and the 4-bit product that need no
GPU: null pointers, sizes, strides, types and alignment are rejected before any
CUDA call; tensors elsewhere than on the current GPU before the library is
called; results are made on the stream of their call."""
import contextlib
import ctypes

import pytest
import torch

import expanded_layout_expert_gb300 as mx
from expanded_layout_expert_gb300 import routing, training, w4
from test_training_devices_host import BF16, Stream, layout, on


@pytest.fixture(scope="module")
def capi():
    from expanded_layout_expert_gb300 import build, _capi
    build.build()
    return _capi


@pytest.fixture(scope="module")
def p():
    buf = (ctypes.c_uint8 * (1 << 16))()
    yield (ctypes.addressof(buf) + 255) // 256 * 256
    del buf


def _refused(capi, rc, text):
    assert rc == capi.MOE_ERR_INVALID_ARG
    got = capi.load().moe_last_error_string().decode()
    assert text in got, got


def test_route_refuses(capi, p):
    f, b = capi.load().moe_route_topk, capi.load().moe_route_topk_backward

    def call(l=p, ld=8, dt=2, bias=None, T=4, E=8, K=2, score=0, ids=p, w=p):
        return f(l, ld, dt, bias, None, T, E, K, score, 0, 1.0, ids, w, None)

    _refused(capi, call(l=None), "null")
    _refused(capi, call(ids=None), "null")
    _refused(capi, call(w=None), "null")
    _refused(capi, call(K=9), "K <= E")
    _refused(capi, call(K=33, E=64, ld=64), "K <= 32")
    _refused(capi, call(E=1025, ld=1025), "E <= 1024")
    _refused(capi, call(K=0), "bad sizes")
    _refused(capi, call(T=-1), "bad sizes")
    _refused(capi, call(dt=3), "dtype")
    _refused(capi, call(score=2), "score")
    _refused(capi, call(ld=7), "stride")
    _refused(capi, call(l=p + 2), "misaligned")
    _refused(capi, call(bias=p + 2), "misaligned")

    def back(dw=p, l=p, ld=8, dt=2, ids=p, T=4, E=8, K=2, score=1, out=p + 4096, ld_o=8):
        return b(dw, l, ld, dt, ids, None, T, E, K, score, 0, 1.0, out, ld_o, None)

    _refused(capi, back(dw=None), "null")
    _refused(capi, back(out=None), "null")
    _refused(capi, back(ld_o=7), "stride")
    _refused(capi, back(dt=5), "dtype")
    _refused(capi, back(score=-1), "score")
    _refused(capi, back(out=p), "must not be logits")
    _refused(capi, back(out=p + 4098), "misaligned")
    _refused(capi, back(K=40, E=64, ld=64, ld_o=64), "K <= 32")


def test_combine_refuses(capi, p):
    f, b = capi.load().moe_combine_rows, capi.load().moe_combine_rows_backward

    def call(rows=p, ld=64, dt=0, src=p, T=4, H=64, K=2, M=8, res=None, ld_r=0, out=p, ld_o=64):
        return f(rows, ld, dt, None, src, None, T, H, K, M, res, ld_r, out, ld_o, None, None)

    _refused(capi, call(rows=None), "null")
    _refused(capi, call(src=None), "null")
    _refused(capi, call(out=None), "null")
    _refused(capi, call(dt=2), "dtype")
    _refused(capi, call(H=60, ld=64), "multiple of 8")
    _refused(capi, call(K=33), "K <= 32")
    _refused(capi, call(ld=56), "strides")
    _refused(capi, call(res=p, ld_r=60), "strides")
    _refused(capi, call(rows=p + 8), "aligned")
    _refused(capi, call(out=p + 4096, res=p + 4096, ld_r=72), "in place")
    _refused(capi, call(), "out must not be rows")

    def back(dy=p, rows=p, ld=64, dt=1, src=p, psum=p, T=4, H=64, K=2, E=4, align=1, M=8, drows=p + 4096, ld_d=64,
             dw=p):
        return b(dy, 64, rows, ld, dt, None, src, psum, None, T, H, K, E, align, M, drows, ld_d, dw, None, None)

    _refused(capi, back(dy=None), "null")
    _refused(capi, back(psum=None), "null")
    _refused(capi, back(rows=None), "null")
    _refused(capi, back(dw=None), "null")
    _refused(capi, back(dt=2), "dtype")
    _refused(capi, back(K=33), "K <= 32")
    _refused(capi, back(align=0), "bad sizes")
    _refused(capi, back(H=12, ld=64), "multiple of 8")
    _refused(capi, back(ld_d=60), "strides")
    _refused(capi, back(drows=p, ld_d=72), "in place")
    _refused(capi, back(drows=p + 4), "aligned")
    _refused(capi, back(E=1 << 20, align=1 << 20), "grid too large")
    _refused(capi, back(drows=p), "drows must not be dy")


def test_w4_refuses(capi, p):
    f = capi.load().moe_grouped_mm_w4

    def call(x=p, ld_x=64, codes=p, scales=p, zeros=None, group=32, start=p, psum=p, dt=0, E=2, N=64, K=64, M=8,
             most=8, out=p, ld=64):
        return f(x, ld_x, codes, scales, zeros, group, start, psum, dt, E, N, K, M, most, out, ld, None, None)

    _refused(capi, call(start=None), "null segments")
    _refused(capi, call(x=None), "non-null")
    _refused(capi, call(codes=None), "non-null")
    _refused(capi, call(scales=None), "non-null")
    _refused(capi, call(dt=2), "dtype")
    _refused(capi, call(group=16), "group")
    _refused(capi, call(group=128), "Kd of the group")
    _refused(capi, call(K=96, group=64, ld_x=96), "Kd of the group")
    _refused(capi, call(N=60, ld=64), "multiple of 8")
    _refused(capi, call(E=1025), "E must be")
    _refused(capi, call(most=9), "max_rows")
    _refused(capi, call(ld_x=56), "row stride")
    _refused(capi, call(ld=60), "row stride")
    _refused(capi, call(x=p + 8), "aligned")
    _refused(capi, call(codes=p + 8), "aligned")
    _refused(capi, call(out=p + 2), "aligned")
    _refused(capi, call(N=1 << 30, K=64, ld=1 << 30, M=1 << 30, most=1 << 30), "32-bit")
    _refused(capi, call(), "out must not be x")


def test_python_refuses():
    l = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="on the GPU"):
        mx.route_topk(l, 2)
    with pytest.raises(ValueError, match="one per 32, 64 or 128"):
        w4._weights(torch.zeros(2, 8, 64, dtype=torch.uint8), torch.zeros(2, 8, 8))
    with pytest.raises(ValueError, match="one per 32, 64 or 128"):
        w4._weights(torch.zeros(2, 8, 64, dtype=torch.uint8), torch.zeros(2, 8, 3))
    with pytest.raises(ValueError):
        w4._weights(torch.zeros(2, 8, 64, dtype=torch.uint8), torch.zeros(2, 8, 0))
    with pytest.raises(ValueError, match="must be"):
        w4._weights(torch.zeros(2, 8, dtype=torch.uint8), torch.zeros(2, 8, 1))
    assert w4._weights(torch.zeros(2, 8, 64, dtype=torch.uint8), torch.zeros(2, 8, 1)) == (2, 8, 128, 128)


# ------------------------------------------------- devices and streams, with stand-ins
F32, I32, U8 = torch.float32, torch.int32, torch.uint8


def arguments():
    """name -> (function, its tensors with their shapes and types, other arguments)"""
    return {
        "route_topk": (routing.route_topk, dict(
            logits=(4, 8, BF16), bias=(8, F32), n_valid=(1, I32), ids=(4, 2, I32), weights=(4, 2, F32)),
            dict(K=2), False),
        "route_topk_backward": (routing.route_topk_backward, dict(
            logits=(4, 8, BF16), dtopk_w=(4, 2, F32), topk_ids=(4, 2, I32), n_valid=(1, I32), out=(4, 8, BF16)),
            {}, False),
        "combine_rows": (routing.combine_rows, dict(
            rows=(8, 16, BF16), topk_w=(4, 2, F32), n_valid=(1, I32), residual=(4, 16, BF16), out=(4, 16, BF16),
            status=(1, I32)), {}, True),
        "combine_rows_backward": (routing.combine_rows_backward, dict(
            dy=(4, 16, BF16), rows=(8, 16, BF16), topk_w=(4, 2, F32), n_valid=(1, I32), drows=(8, 16, BF16),
            dtopk_w=(4, 2, F32), status=(1, I32)), {}, True),
        "grouped_matmul_w4": (w4.grouped_matmul_w4, dict(
            x=(8, 32, BF16), codes=(2, 24, 16, U8), scales=(2, 24, 1, BF16), zeros=(2, 24, 1, U8),
            out=(8, 24, BF16), status=(1, I32)), {}, True),
    }


@pytest.fixture
def calls(monkeypatch):
    got = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: got.append(name) or 0

    for module in (routing, w4):
        monkeypatch.setattr(module, "load", Library)
    monkeypatch.setattr(training, "_current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    return got


@pytest.mark.parametrize("name", arguments())
def test_devices(calls, name):
    f, shapes, more, takes_lay = arguments()[name]

    def call(lay=0, stream=None, **where):
        kw = {k: on(where.get(k, where.get("all", 0)), *s[:-1], dtype=s[-1]) for k, s in shapes.items()}
        if takes_lay:
            kw["lay"] = layout(lay)
        return f(**kw, **more, stream=stream)

    call()
    call(stream=Stream(0))
    assert len(calls) == 2
    for k in shapes:
        for gpu in (1, -1):
            with pytest.raises(ValueError):
                call(**{k: gpu})
    wrong = [dict(all=1, lay=1), dict(all=1, lay=1, stream=Stream(1)), dict(stream=Stream(1))]
    for kw in wrong + ([dict(lay=1)] if takes_lay else []):
        with pytest.raises(ValueError):
            call(**kw)
    assert len(calls) == 2


@pytest.mark.parametrize("name", arguments())
def test_wrong_shapes_and_types(calls, name):
    f, shapes, more, takes_lay = arguments()[name]
    for k, s in shapes.items():
        if s[:-1] == (1,):
            continue
        if k == "logits" or (k, name) in (("rows", "combine_rows"), ("x", "grouped_matmul_w4")):
            bad = [(*s[:-1], torch.float64)]
        else:
            bad = [(*s[:-2], s[-2] + 8, s[-1]), (*s[:-1], torch.float64)]
        for b in bad:
            kw = {n: on(0, *(b if n == k else v)[:-1], dtype=(b if n == k else v)[-1]) for n, v in shapes.items()}
            if takes_lay:
                kw["lay"] = layout(0)
            with pytest.raises(ValueError):
                f(**kw, **more)
    assert not calls


def test_unknown_score(calls):
    with pytest.raises(ValueError, match="score"):
        routing.route_topk(on(0, 4, 8), 2, score="relu")
    assert not calls


@pytest.mark.parametrize("name", arguments())
def test_results_are_made_on_the_calls_stream(monkeypatch, name):
    current, seen = [None], []

    @contextlib.contextmanager
    def stream(s):
        was, current[0] = current[0], s
        yield
        current[0] = was

    def recorded(make):
        def g(*a, **k):
            seen.append(current[0])
            return make(*a, **k)
        return g

    f, shapes, more, takes_lay = arguments()[name]
    made = {"ids", "weights", "out", "drows"} | ({"dtopk_w"} if name == "combine_rows_backward" else set())
    kw = {k: torch.ones(*s[:-1]).to(s[-1]) for k, s in shapes.items() if k not in made}
    if takes_lay:
        i32 = lambda *s: torch.ones(*s, dtype=I32)  # noqa: E731
        kw["lay"] = mx.Layout(psum=i32(2), start=i32(2), total=i32(1), m_indices=i32(8), src2dst=i32(4, 2),
                              tile_prefix=i32(3), E=2, align=1, M_cap=8)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    for n in ("zeros", "empty"):
        monkeypatch.setattr(torch, n, recorded(getattr(torch, n)))
    for module in (routing, w4):
        monkeypatch.setattr(module, "load", type("L", (), {"__getattr__": lambda s, n: lambda *a: 0}))
        for n in ("_rows", "_whole", "_word", "_stream", "_device"):
            monkeypatch.setattr(module, n, (lambda t, *a: (0, t.shape[1])) if n == "_rows" else (lambda *a: 0))
    monkeypatch.setattr(training, "_whole", lambda *a: 0)
    for side in (object(), None):
        seen.clear()
        f(**kw, **more, stream=side)
        assert seen and all(s is side for s in seen)


def test_kernels_do_not_spill():
    from expanded_layout_expert_gb300 import build
    for src in ("route.cu", "combine_rows.cu", "grouped_w4.cu", "grouped_w4_few.cu"):
        allowed = 8 if src == "grouped_w4_few.cu" else 0   # a value outside the loop
        for name, v in build.ptxas_usage(src).items():
            assert v["spill_st"] <= allowed and v["stack"] <= allowed, (name, v)
