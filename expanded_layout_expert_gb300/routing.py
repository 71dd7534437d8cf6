"""The layer's two ends: the top-k router and the weighted return of the
experts' rows to their tokens, each with its gradient (bindings of
moe_route_topk, moe_combine_rows and their backward calls in
include/moe_expand.h).

The functions marshal as those of ``training`` do: tensors and a given stream
are on the current GPU, row tensors may have a row stride, and results that a
call makes itself are made on the stream it is queued on.
"""
from __future__ import annotations

from typing import Optional

import torch

from ._capi import MOE_SCORE_SIGMOID, MOE_SCORE_SOFTMAX, check, load
from .training import TYPE_CODE, _code16, _device, _new, _rows, _stream, _whole, _word

__all__ = ["route_topk", "route_topk_backward", "combine_rows", "combine_rows_backward"]

_SCORES = {"softmax": MOE_SCORE_SOFTMAX, "sigmoid": MOE_SCORE_SIGMOID}


def _score(score: str) -> int:
    if score not in _SCORES:
        raise ValueError(f"score must be 'softmax' or 'sigmoid', got {score!r}")
    return _SCORES[score]


def _logits(t: torch.Tensor, name: str, T: int, E: int, dtype, dev: int) -> tuple:
    """(pointer, row stride, type code) of a [T, E] tensor with contiguous rows."""
    if t.dtype not in TYPE_CODE:
        raise ValueError(f"{name} must be float32, bfloat16 or float16, got {t.dtype}")
    ptr, ld = _rows(t, name, T, E, dtype, dev)
    return ptr, ld, TYPE_CODE[t.dtype]


def route_topk(logits: torch.Tensor, K: int, *, score: str = "softmax", renormalize: bool = False,
               factor: float = 1.0, bias: Optional[torch.Tensor] = None,
               n_valid: Optional[torch.Tensor] = None, ids: Optional[torch.Tensor] = None,
               weights: Optional[torch.Tensor] = None, stream=None):
    """(topk_ids int32 [T, K], topk_w float32 [T, K]) of the router's logits
    [T, E] (float32, bfloat16 or float16): the K largest of logit + bias, ties to
    the lowest expert, with weights ``factor`` times their softmax over all
    experts or their sigmoid; ``renormalize``: over the chosen alone. ``bias``
    (float32 [E]) moves the choice, not the weights. Experts at -inf (or NaN) are
    never chosen: id -1 and weight 0 where fewer than K are left. Rows t >=
    n_valid are neither read nor written (ids made here hold -1 there)."""
    T, E = logits.shape
    dev = _device(logits, "logits")
    lp, ld, dt = _logits(logits, "logits", T, E, logits.dtype, dev)
    code = _score(score)
    if ids is None:
        ids = _new(torch.empty, (T, K), torch.int32, logits, stream)
        if n_valid is not None:
            with torch.cuda.stream(stream):
                ids.fill_(-1)
    else:
        _whole(ids, "ids", (T, K), torch.int32, dev)
    if weights is None:
        weights = _new(torch.empty if n_valid is None else torch.zeros, (T, K), torch.float32, logits, stream)
    else:
        _whole(weights, "weights", (T, K), torch.float32, dev)
    rc = load().moe_route_topk(
        lp, ld, dt, _whole(bias, "bias", (E,), torch.float32, dev), _word(n_valid, "n_valid", dev), T, E, K,
        code, int(renormalize), factor, ids.data_ptr(), weights.data_ptr(), _stream(stream, dev))
    check(rc, "moe_route_topk")
    return ids, weights


def route_topk_backward(dtopk_w: torch.Tensor, logits: torch.Tensor, topk_ids: torch.Tensor, *,
                        score: str = "softmax", renormalize: bool = False, factor: float = 1.0,
                        n_valid: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                        stream=None) -> torch.Tensor:
    """The gradient of route_topk's logits, in their type, from that of its
    weights and the ids it chose, with the same score, renormalize and factor.
    Every entry of the rows t < n_valid is written."""
    T, E = logits.shape
    K = topk_ids.shape[1]
    dev = _device(logits, "logits")
    lp, ld, dt = _logits(logits, "logits", T, E, logits.dtype, dev)
    code = _score(score)
    if out is None:
        out = _new(torch.empty if n_valid is None else torch.zeros, (T, E), logits.dtype, logits, stream)
    op, ld_o, _ = _logits(out, "out", T, E, logits.dtype, dev)
    rc = load().moe_route_topk_backward(
        _whole(dtopk_w, "dtopk_w", (T, K), torch.float32, dev), lp, ld, dt,
        _whole(topk_ids, "topk_ids", (T, K), torch.int32, dev), _word(n_valid, "n_valid", dev), T, E, K, code,
        int(renormalize), factor, op, ld_o, _stream(stream, dev))
    check(rc, "moe_route_topk_backward")
    return out


def combine_rows(rows: torch.Tensor, lay, topk_w: Optional[torch.Tensor] = None,
                 n_valid: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """out[t] = residual[t] + sum_k topk_w[t, k] * rows[src2dst[t, k]] over the
    token's pairs (residual None: 0, topk_w None: 1); bfloat16 or float16.
    ``out`` may be ``residual``. Rows t >= n_valid are not written."""
    T, K = lay.src2dst.shape
    H = rows.shape[1]
    dt, dev = _code16(rows, "rows"), _device(rows, "rows")
    if out is None:
        out = _new(torch.empty if n_valid is None else torch.zeros, (T, H), rows.dtype, rows, stream)
    rp, ld_r = _rows(rows, "rows", lay.M_cap, H, rows.dtype, dev)
    sp, ld_s = (None, 0) if residual is None else _rows(residual, "residual", T, H, rows.dtype, dev)
    op, ld_o = _rows(out, "out", T, H, rows.dtype, dev)
    rc = load().moe_combine_rows(
        rp, ld_r, dt, _whole(topk_w, "topk_w", (T, K), torch.float32, dev),
        _whole(lay.src2dst, "lay.src2dst", (T, K), torch.int32, dev), _word(n_valid, "n_valid", dev), T, H, K,
        lay.M_cap, sp, ld_s, op, ld_o, _word(status, "status", dev), _stream(stream, dev))
    check(rc, "moe_combine_rows")
    return out


def combine_rows_backward(dy: torch.Tensor, rows: torch.Tensor, lay,
                          topk_w: Optional[torch.Tensor] = None,
                          n_valid: Optional[torch.Tensor] = None, drows: Optional[torch.Tensor] = None,
                          dtopk_w: Optional[torch.Tensor] = None,
                          status: Optional[torch.Tensor] = None, stream=None):
    """(drows [M_cap, H], dtopk_w [T, K]): the gradients of combine_rows' rows
    and weights; that of its residual is dy. Alignment gaps of drows are zeroed.
    ``drows`` may be ``rows`` itself, which is then overwritten."""
    T, K = lay.src2dst.shape
    H = dy.shape[1]
    dt, dev = _code16(dy, "dy"), _device(dy, "dy")
    if drows is None:
        drows = _new(torch.zeros, (lay.M_cap, H), dy.dtype, dy, stream)
    if dtopk_w is None:
        dtopk_w = _new(torch.empty if n_valid is None else torch.zeros, (T, K), torch.float32, dy, stream)
    yp, ld_y = _rows(dy, "dy", T, H, dy.dtype, dev)
    rp, ld_r = _rows(rows, "rows", lay.M_cap, H, dy.dtype, dev)
    dp, ld_d = _rows(drows, "drows", lay.M_cap, H, dy.dtype, dev)
    rc = load().moe_combine_rows_backward(
        yp, ld_y, rp, ld_r, dt, _whole(topk_w, "topk_w", (T, K), torch.float32, dev),
        _whole(lay.src2dst, "lay.src2dst", (T, K), torch.int32, dev),
        _whole(lay.psum, "lay.psum", (lay.E,), torch.int32, dev), _word(n_valid, "n_valid", dev), T, H, K,
        lay.E, lay.align, lay.M_cap, dp, ld_d, _whole(dtopk_w, "dtopk_w", (T, K), torch.float32, dev),
        _word(status, "status", dev), _stream(stream, dev))
    check(rc, "moe_combine_rows_backward")
    return drows, dtopk_w
