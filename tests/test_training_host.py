"""Refusals of the training calls that need no GPU: null pointers, sizes,
strides, types and alignment are rejected before any CUDA call, with a message."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def capi():
    from expanded_layout_expert_gb300 import build, _capi
    build.build()
    return _capi


@pytest.fixture(scope="module")
def p():
    buf = (ctypes.c_uint8 * (1 << 16))()
    a = ctypes.addressof(buf)
    yield (a + 255) // 256 * 256
    del buf


def _refused(capi, rc, text):
    assert rc == capi.MOE_ERR_INVALID_ARG
    got = capi.load().moe_last_error_string().decode()
    assert text in got, got


def test_expand_rows_refuses(capi, p):
    f = capi.load().moe_expand_rows

    def call(x=p, ld_x=64, w=None, src=p, psum=p, T=4, H=64, K=2, E=4, align=1, M=8, xe=p, ld=64,
             row_w=None):
        return f(x, ld_x, w, src, psum, None, T, H, K, E, align, M, xe, ld, row_w, None, None)

    _refused(capi, call(x=None), "null")
    _refused(capi, call(psum=None), "null")
    _refused(capi, call(H=60, ld_x=60, ld=60), "multiple of 8")
    _refused(capi, call(ld_x=56), "strides")
    _refused(capi, call(ld=68), "strides")
    _refused(capi, call(K=33), "K <= 32")
    _refused(capi, call(align=0), "bad sizes")
    _refused(capi, call(x=p + 2), "aligned")
    _refused(capi, call(row_w=p), "topk_w")


def test_collect_row_grads_refuses(capi, p):
    f = capi.load().moe_collect_row_grads
    _refused(capi, f(p, p, None, 4, 33, 8, p, None), "K <= 32")
    _refused(capi, f(p, None, None, 4, 2, 8, p, None), "null")
    _refused(capi, f(None, p, None, 4, 2, 8, p, None), "null")


@pytest.mark.parametrize("which", ["moe_grouped_mm", "moe_grouped_mm_dgrad"])
def test_grouped_mm_refuses(capi, p, which):
    f = getattr(capi.load(), which)

    def call(x=p, ld_x=64, w=p, start=p, psum=p, dt=capi.MOE_BF16, E=2, N=64, K=64, M=8, most=None,
             out=p, ld=64):
        return f(x, ld_x, w, start, psum, dt, E, N, K, M, M if most is None else most, out, ld, None, None)

    _refused(capi, call(most=9), "max_rows")
    _refused(capi, call(most=-1), "max_rows")

    _refused(capi, call(x=None), "non-null")
    _refused(capi, call(w=None), "non-null")
    _refused(capi, call(psum=None), "null segments")
    _refused(capi, call(dt=capi.MOE_F32), "dtype")
    _refused(capi, call(dt=7), "dtype")
    _refused(capi, call(E=0), "E must be")
    _refused(capi, call(E=1025), "E must be")
    _refused(capi, call(N=60), "multiples of 8")
    _refused(capi, call(K=0), "multiples of 8")
    _refused(capi, call(ld_x=56), "row stride")
    _refused(capi, call(ld=65), "row stride")
    _refused(capi, call(x=p + 8), "aligned")
    _refused(capi, call(out=p + 2), "aligned")
    _refused(capi, call(M=-1), "M_cap")
    _refused(capi, call(N=1 << 20, K=1 << 20, M=1 << 30, ld=1 << 20, ld_x=1 << 20), "32-bit")


def test_wgrad_refuses(capi, p):
    f = capi.load().moe_grouped_mm_wgrad

    def call(dy=p, ld_dy=64, x=p, ld_x=64, start=p, psum=p, dt=capi.MOE_BF16, E=2, N=64, K=64, M=8,
             dw=p, out=capi.MOE_F32, acc=0):
        return f(dy, ld_dy, x, ld_x, start, psum, dt, E, N, K, M, dw, out, acc, None, None)

    _refused(capi, call(dy=None), "non-null")
    _refused(capi, call(dw=None), "non-null")
    _refused(capi, call(start=None), "null segments")
    _refused(capi, call(out=capi.MOE_F16), "operands' type")
    _refused(capi, call(dt=capi.MOE_F32), "dtype")
    _refused(capi, call(N=4), "multiples of 8")
    _refused(capi, call(ld_dy=60), "row stride")
    _refused(capi, call(dw=p + 4), "aligned")


def test_swiglu_refuses(capi, p):
    f, b = capi.load().moe_swiglu, capi.load().moe_swiglu_backward

    def call(gu=p, ld=128, dt=capi.MOE_BF16, I=64, total=p, M=4, h=p, ld_h=64):
        return f(gu, ld, dt, I, None, total, M, h, ld_h, None)

    _refused(capi, call(gu=None), "null")
    _refused(capi, call(total=None), "null")
    _refused(capi, call(dt=capi.MOE_F32), "dtype")
    _refused(capi, call(I=12), "multiple of 8")
    _refused(capi, call(ld=120), "strides")
    _refused(capi, call(h=p + 8), "aligned")

    def back(dh=p, ld_dh=64, gu=p, ld=128, dt=capi.MOE_BF16, I=64, dgu=p + 4096, ld_dgu=128):
        return b(dh, ld_dh, gu, ld, dt, I, None, p, 4, dgu, ld_dgu, None, None)

    _refused(capi, back(dh=None), "null")
    _refused(capi, back(ld_dgu=64), "strides")
    _refused(capi, back(dgu=p, ld_dgu=136), "in place")
    _refused(capi, back(dgu=p + 8), "aligned")


def test_adamw_refuses(capi, p):
    import numpy as np
    from expanded_layout_expert_gb300.training import _ADAMW_TENSOR
    assert _ADAMW_TENSOR.itemsize == 80
    f = capi.load().moe_adamw_step

    def call(bits=32, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, wd=0.0, step=1, count=1, **kw):
        t = np.zeros(1, dtype=_ADAMW_TENSOR)
        for k, v in dict(dict(p=p, g=p, m=p, v=p, m_scale=p, v_scale=p, n=4, p_type=2, g_type=2),
                         **kw).items():
            t[k] = 0 if v is None else v
        return f(t.ctypes.data, count, bits, lr, b1, b2, eps, wd, step, None, None)

    _refused(capi, call(bits=16), "state_bits")
    _refused(capi, call(step=0), "step")
    _refused(capi, call(b1=1.0), "betas")
    _refused(capi, call(b2=-0.1), "betas")
    _refused(capi, call(eps=-1.0), "eps")
    _refused(capi, call(lr=float("nan")), "finite")
    _refused(capi, call(count=-1), "null")
    _refused(capi, call(n=-1), "negative")
    _refused(capi, call(g=None), "null")
    _refused(capi, call(bits=8, m_scale=None), "null")
    _refused(capi, call(p_type=3), "type")
    _refused(capi, call(p=p + 2), "aligned")
    assert f(None, 0, 32, 1e-3, 0.9, 0.99, 1e-8, 0.0, 1, None, None) in (
        capi.MOE_OK, capi.MOE_ERR_UNSUPPORTED)   # nothing to do


def test_grouped_product_kernels_keep_their_registers():
    """wgrad's warps trade registers (setmaxnreg): 56 * 128 + 224 * 256 must be
    exactly what the block of 384 threads is launched with, or the claim would
    wait for registers that never come. Spills: at most twelve words, once a
    tile; none in the kernels without a trade."""
    from expanded_layout_expert_gb300 import build
    wgrad = 0
    for name, v in build.ptxas_usage("grouped_mm16.cu").items():
        if "grouped_mm16_kernelILi2E" in name:
            wgrad += 1
            assert v["registers"] * 384 == 56 * 128 + 224 * 256, (name, v)
            assert v["spill_st"] <= 48, (name, v)
        else:
            assert v["spill_st"] == 0 and v["stack"] == 0, (name, v)
    assert wgrad == 16   # type x result type x added or not x CTAs a tile
    for src in ("grouped_mm16_few.cu", "adamw.cu", "swiglu.cu", "expand_rows.cu"):
        for name, v in build.ptxas_usage(src).items():
            assert v["spill_st"] == 0, (name, v)
