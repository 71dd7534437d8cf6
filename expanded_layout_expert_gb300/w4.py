"""The experts in 4 bits, for batches of single tokens: the grouped product over
4-bit weights with group scales (moe_grouped_mm_w4 of include/moe_expand.h), and
the layer of it.

Weights: codes uint8 [E, N, Kd / 2], the value of an even k in a byte's low four
bits and that of k + 1 in its high ones; scales [E, N, Kd / group] in the
activations' type; zero points uint8 [E, N, Kd / group] of 0 to 15, or None for 8
everywhere. A weight is scale * (code - zero point).
"""
from __future__ import annotations

from typing import Optional

import torch

from ._capi import check, load
from .training import (_code16, _device, _most_rows, _new, _rows, _segments, _stream, _whole, _word,
                       expand_rows, swiglu)

__all__ = ["grouped_matmul_w4", "FourBitExperts"]

GROUPS = (32, 64, 128)


def _weights(codes: torch.Tensor, scales: torch.Tensor) -> tuple:
    """(E, N, Kd, group) of codes [E, N, Kd / 2] and scales [E, N, Kd / group]."""
    if codes.dim() != 3 or scales.dim() != 3:
        raise ValueError("codes must be [E, N, Kd / 2] and scales [E, N, Kd / group]")
    E, N, half = codes.shape
    G = scales.shape[2]
    group = 2 * half // G if G else 0
    if group not in GROUPS or group * G != 2 * half:
        raise ValueError(f"{G} scales for {2 * half} values: one per 32, 64 or 128 is needed")
    return E, N, 2 * half, group


def grouped_matmul_w4(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, lay,
                      zeros: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                      status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out[r] = x[r] @ w[e].T for the rows r of expert e, w[e] = scales * (codes -
    zeros); x [M, Kd], out [M, N], bfloat16 or float16. Made for few rows per
    expert, right for any number: from some 96 to 192 of them on (groups of 32: 48 to
    96) grouped_matmul over 16-bit weights is the faster call."""
    dt, dev = _code16(x, "x"), _device(x, "x")
    start, psum, E = _segments(lay, dev)
    _, N, Kd, group = _weights(codes, scales)
    M = x.shape[0]
    if out is None:
        out = _new(torch.zeros, (M, N), x.dtype, x, stream)
    xp, ld_x = _rows(x, "x", M, Kd, x.dtype, dev)
    op, ld_o = _rows(out, "out", M, N, x.dtype, dev)
    G = Kd // group
    rc = load().moe_grouped_mm_w4(
        xp, ld_x, _whole(codes, "codes", (E, N, Kd // 2), torch.uint8, dev),
        _whole(scales, "scales", (E, N, G), x.dtype, dev), _whole(zeros, "zeros", (E, N, G), torch.uint8, dev),
        group, start, psum, dt, E, N, Kd, M, _most_rows(lay, M), op, ld_o, _word(status, "status", dev),
        _stream(stream, dev))
    check(rc, "moe_grouped_mm_w4")
    return out


class FourBitExperts:
    """The experts of an expanded-layout MoE layer in 4 bits, for decode batches of
    up to ``max_tokens`` tokens; every buffer allocated once.

        forward(x, topk_ids, topk_w, n_valid, residual) -> y [T, H]

    y[t] = residual[t] + sum_k w[t, k] * w2[e] (silu(g) * u), [g | u] = w13[e]
    x[t], e = topk_ids[t, k] (route_topk gives ids and weights). w13 and w2 are
    (codes, scales, zero points or None) of [E, 2I, H] and [E, H, I] weights as
    grouped_matmul_w4 takes them; x, y, residual and the scales are all bfloat16 or
    all float16. The intermediate rows are rounded to that type once per product.
    Rows t >= n_valid are neither read nor written. Call it within a CUDA graph for
    the smallest batches, after one call outside.

    What is launched goes by ``max_tokens``, not by n_valid, which only the device
    knows: 8 tokens of 8 out of 64 experts (H = 4096, I = 2048) take 141 us in a layer
    for 8 and 162 in one for 256. So make one for each batch size that is captured. Its
    buffers are one set: two forwards, or graphs of them, are not to run at once.
    """

    def __init__(self, w13, w2, *, K: int, max_tokens: int, align: int = 1):
        from . import Layout, expanded_capacity, workspace_size
        weights = []
        for name, w in (("w13", w13), ("w2", w2)):
            codes, scales, zeros = w
            E, N, Kd, group = _weights(codes, scales)
            _code16(scales, f"{name}'s scales")
            dev = codes.get_device()
            if dev < 0:
                raise ValueError(f"{name} must be on the GPU")
            _whole(codes, f"{name}'s codes", (E, N, Kd // 2), torch.uint8, dev)
            _whole(scales, f"{name}'s scales", (E, N, Kd // group), scales.dtype, dev)
            _whole(zeros, f"{name}'s zero points", (E, N, Kd // group), torch.uint8, dev)
            weights.append((E, N, Kd, dev, scales.dtype))
        (E, twoI, H, dev, dtype), second = weights
        if twoI % 2 or second != (E, H, twoI // 2, dev, dtype):
            raise ValueError("w13 must be [E, 2I, H] and w2 [E, H, I], on one GPU, with scales of one type")
        self.w13, self.w2 = tuple(w13), tuple(w2)
        self.E, self.H, self.I, self.K, self.align, self.T = E, H, twoI // 2, K, align, max_tokens
        self.dtype = dtype
        device = w13[0].device
        M = self.M_cap = max(1, expanded_capacity(max_tokens, K, E, align))
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=device)  # noqa: E731
        b16 = lambda *s: torch.zeros(*s, dtype=dtype, device=device)  # noqa: E731
        self.ws = torch.zeros(workspace_size(max_tokens, K, E), dtype=torch.uint8, device=device)
        self.status = i32(1)
        self.lay = Layout(psum=i32(E), start=i32(E), total=i32(1), m_indices=i32(M),
                          src2dst=i32(max_tokens, K), tile_prefix=i32(E + 1), E=E, align=align, M_cap=M)
        self.xe, self.gu, self.h, self.down = b16(M, H), b16(M, twoI), b16(M, self.I), b16(M, H)
        self.y = b16(max_tokens, H)

    def forward(self, x: torch.Tensor, topk_ids: torch.Tensor, topk_w: torch.Tensor,
                n_valid: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """y (self.y, or ``out``: [T, H]; it may be ``residual``)."""
        from . import combine_rows, expand_layout
        dev = _device(self.w13[0], "w13")
        y = self.y if out is None else out
        for name, t in (("x", x), ("out", y)) + ((("residual", residual),) if residual is not None else ()):
            _rows(t, name, self.T, self.H, self.dtype, dev)
        _whole(topk_ids, "topk_ids", (self.T, self.K), torch.int32, dev)
        if _whole(topk_w, "topk_w", (self.T, self.K), torch.float32, dev) is None:
            raise ValueError("topk_w is needed")
        _word(n_valid, "n_valid", dev)
        _stream(stream, dev)
        lay, st = self.lay, self.status
        expand_layout(topk_ids, self.E, self.align, self.M_cap, n_valid, self.ws, st, lay, stream)
        expand_rows(x, lay, None, n_valid, self.xe, None, st, stream)
        codes, scales, zeros = self.w13
        grouped_matmul_w4(self.xe, codes, scales, lay, zeros, self.gu, st, stream)
        swiglu(self.gu, lay, None, self.h, stream)
        codes, scales, zeros = self.w2
        grouped_matmul_w4(self.h, codes, scales, lay, zeros, self.down, st, stream)
        return combine_rows(self.down, lay, topk_w, n_valid, residual, y, st, stream)
