"""The experts in 4 bits, for batches of single tokens: the grouped product over
4-bit weights with group scales (moe_grouped_mm_w4 of include/moe_expand.h).

Weights: codes uint8 [E, N, Kd / 2], the value of an even k in a byte's low four
bits and that of k + 1 in its high ones; scales [E, N, Kd / group] in the
activations' type; zero points uint8 [E, N, Kd / group] of 0 to 15, or None for 8
everywhere. A weight is scale * (code - zero point).
"""
from __future__ import annotations

from typing import Optional

import torch

from ._capi import check, load
from .training import _code16, _device, _most_rows, _new, _rows, _segments, _stream, _whole, _word

__all__ = ["grouped_matmul_w4"]

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
    expert; right for any number."""
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
