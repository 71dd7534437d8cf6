"""Training the experts in 16 bits over the expanded layout: bindings of the
training calls of include/moe_expand.h, and the layer that strings them
together.

Each function marshals torch tensors and the current CUDA stream into one C
call, as the package's other functions do. All tensors of a call, and a stream
given to it, are on the current GPU; others are refused. Row tensors may have a
row stride larger than the row (a multiple of 8 values); rows outside the
segments [start[e], psum[e]) of the layout are neither used nor written. A
result that a call makes itself is made on the stream the call is queued on.
"""
from __future__ import annotations

from typing import List, Optional, Sequence

import numpy as np
import torch

from ._capi import MOE_BF16, MOE_F16, MOE_F32, check, load

__all__ = ["expand_rows", "collect_row_grads", "grouped_matmul", "grouped_matmul_dgrad",
           "grouped_matmul_wgrad", "swiglu", "swiglu_backward", "AdamW", "TrainableExperts"]

TYPE_CODE = {torch.bfloat16: MOE_BF16, torch.float16: MOE_F16, torch.float32: MOE_F32}
STATE_BLOCK = 128   # values that share a scale in an 8-bit AdamW state


def _current_device() -> int:
    return torch._C._cuda_getDevice()


def _device(t: torch.Tensor, name: str) -> int:
    """Index of the GPU a call runs on: that of its first tensor, which must be
    the current one, because the library launches there. The call's other
    tensors and its stream are held against it."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be on the GPU")
    if dev != _current_device():
        raise ValueError(f"{name} is on GPU {dev}, but the current one is {_current_device()}: enter its "
                         "device first")
    return dev


def _stream(stream, dev: int):
    """The given stream's handle, or that of the device's current stream
    (without building a stream object for it)."""
    if stream is not None:
        if stream.device_index != dev:
            raise ValueError(f"the stream is on GPU {stream.device_index}, the tensors on {dev}")
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(dev)


def _new(make, shape: tuple, dtype, like: torch.Tensor, stream) -> torch.Tensor:
    """A result tensor, made by torch.zeros or torch.empty on the stream that
    fills it: zeroed on another one it could be wiped after the kernel, and
    its memory given away while the kernel still writes."""
    if stream is None:
        return make(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return make(shape, dtype=dtype, device=like.device)


def _code16(t: torch.Tensor, name: str) -> int:
    if t.dtype is torch.bfloat16:
        return MOE_BF16
    if t.dtype is torch.float16:
        return MOE_F16
    raise ValueError(f"{name} must be bfloat16 or float16, got {t.dtype}")


def _rows(t: torch.Tensor, name: str, rows: int, width: int, dtype, dev: int) -> tuple:
    """(pointer, row stride) of a [rows, width] tensor with contiguous rows."""
    if t.shape != (rows, width):
        raise ValueError(f"{name} must be [{rows}, {width}], got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    ld, one = t.stride()
    if rows <= 1:
        ld = width   # one row has no stride to speak of
    if (one != 1 and width > 1) or ld < width:
        raise ValueError(f"{name} must have contiguous, non-overlapping rows")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on GPU {dev}")
    return t.data_ptr(), ld


def _whole(t: Optional[torch.Tensor], name: str, shape: tuple, dtype, dev: int):
    """Pointer of a contiguous tensor of the given shape and type (None: NULL)."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dtype or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on GPU {dev}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _word(t: Optional[torch.Tensor], name: str, dev: int):
    if t is None:
        return None
    if t.dtype is not torch.int32 or t.numel() < 1 or t.get_device() != dev:
        raise ValueError(f"{name} must be an int32 tensor of one element on GPU {dev}")
    return t.data_ptr()


def _segments(lay, dev: int) -> tuple:
    E = lay.E
    return _whole(lay.start, "lay.start", (E,), torch.int32, dev), \
        _whole(lay.psum, "lay.psum", (E,), torch.int32, dev), E


def _most_rows(lay, M: int) -> int:
    """Rows of all segments together, at most: one per pair of the layout (a
    layout without pairs of its own may fill the buffer)."""
    pairs = lay.src2dst.numel()
    return min(pairs, M) if pairs else M


def expand_rows(x: torch.Tensor, lay, topk_w: Optional[torch.Tensor] = None,
                n_valid: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                row_w: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                stream=None):
    """16-bit rows of the valid pairs: out[src2dst[t, k]] = x[t], alignment
    gaps zeroed. With ``topk_w`` also row_w[src2dst[t, k]] = topk_w[t, k] and
    (out, row_w) is returned, else out."""
    T, H = x.shape
    K = lay.src2dst.shape[1]
    _code16(x, "x")
    dev = _device(x, "x")
    if out is None:
        out = _new(torch.zeros, (lay.M_cap, H), x.dtype, x, stream)
    if topk_w is not None and row_w is None:
        row_w = _new(torch.zeros, (lay.M_cap,), torch.float32, x, stream)
    if topk_w is None and row_w is not None:
        raise ValueError("row_w needs topk_w")
    xp, ld_x = _rows(x, "x", T, H, x.dtype, dev)
    op, ld_o = _rows(out, "out", lay.M_cap, H, x.dtype, dev)
    rc = load().moe_expand_rows(
        xp, ld_x, _whole(topk_w, "topk_w", (T, K), torch.float32, dev),
        _whole(lay.src2dst, "lay.src2dst", (T, K), torch.int32, dev),
        _whole(lay.psum, "lay.psum", (lay.E,), torch.int32, dev), _word(n_valid, "n_valid", dev), T, H,
        K, lay.E, lay.align, lay.M_cap, op, ld_o,
        _whole(row_w, "row_w", (lay.M_cap,), torch.float32, dev), _word(status, "status", dev),
        _stream(stream, dev))
    check(rc, "moe_expand_rows")
    return out if topk_w is None else (out, row_w)


def collect_row_grads(rows: torch.Tensor, lay, n_valid: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Per-row values back to their pairs: out[t, k] = rows[src2dst[t, k]], 0
    where there is no pair (the gradient of the top-k weights)."""
    T, K = lay.src2dst.shape
    dev = _device(rows, "rows")
    if out is None:
        out = _new(torch.zeros, (T, K), torch.float32, rows, stream)
    rc = load().moe_collect_row_grads(
        _whole(rows, "rows", (lay.M_cap,), torch.float32, dev),
        _whole(lay.src2dst, "lay.src2dst", (T, K), torch.int32, dev), _word(n_valid, "n_valid", dev), T, K,
        lay.M_cap, _whole(out, "out", (T, K), torch.float32, dev), _stream(stream, dev))
    check(rc, "moe_collect_row_grads")
    return out


def grouped_matmul(x: torch.Tensor, w: torch.Tensor, lay, out: Optional[torch.Tensor] = None,
                   status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out[r] = x[r] @ w[e].T for the rows r of expert e; x [M, Kd], w
    [E, N, Kd], out [M, N], all bfloat16 or all float16."""
    dt, dev = _code16(x, "x"), _device(x, "x")
    start, psum, E = _segments(lay, dev)
    M, Kd = x.shape
    N = w.shape[1]
    if out is None:
        out = _new(torch.zeros, (M, N), x.dtype, x, stream)
    xp, ld_x = _rows(x, "x", M, Kd, x.dtype, dev)
    op, ld_o = _rows(out, "out", M, N, x.dtype, dev)
    rc = load().moe_grouped_mm(xp, ld_x, _whole(w, "w", (E, N, Kd), x.dtype, dev), start, psum, dt, E, N,
                               Kd, M, _most_rows(lay, M), op, ld_o, _word(status, "status", dev),
                               _stream(stream, dev))
    check(rc, "moe_grouped_mm")
    return out


def grouped_matmul_dgrad(dy: torch.Tensor, w: torch.Tensor, lay, out: Optional[torch.Tensor] = None,
                         status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The gradient of grouped_matmul's x: out[r] = dy[r] @ w[e]; dy [M, N],
    out [M, Kd]."""
    dt, dev = _code16(dy, "dy"), _device(dy, "dy")
    start, psum, E = _segments(lay, dev)
    M, N = dy.shape
    Kd = w.shape[2]
    if out is None:
        out = _new(torch.zeros, (M, Kd), dy.dtype, dy, stream)
    dp, ld_d = _rows(dy, "dy", M, N, dy.dtype, dev)
    op, ld_o = _rows(out, "out", M, Kd, dy.dtype, dev)
    rc = load().moe_grouped_mm_dgrad(dp, ld_d, _whole(w, "w", (E, N, Kd), dy.dtype, dev), start, psum, dt,
                                     E, N, Kd, M, _most_rows(lay, M), op, ld_o,
                                     _word(status, "status", dev), _stream(stream, dev))
    check(rc, "moe_grouped_mm_dgrad")
    return out


def grouped_matmul_wgrad(dy: torch.Tensor, x: torch.Tensor, lay, out: Optional[torch.Tensor] = None,
                         accumulate: bool = False, out_dtype=None,
                         status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The gradient of grouped_matmul's w: out[e] = dy[rows of e].T @ x[rows of
    e], in the operands' type or float32 (``out_dtype``); ``accumulate`` adds
    it to what ``out`` holds, rounded once."""
    dt, dev = _code16(dy, "dy"), _device(dy, "dy")
    start, psum, E = _segments(lay, dev)
    M, N = dy.shape
    Kd = x.shape[1]
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out = _new(torch.empty, (E, N, Kd), out_dtype or dy.dtype, dy, stream)
    elif out_dtype is not None and out.dtype is not out_dtype:
        raise ValueError(f"out must be {out_dtype}, got {out.dtype}")
    if out.dtype is not dy.dtype and out.dtype is not torch.float32:
        raise ValueError(f"out must be {dy.dtype} or float32, got {out.dtype}")
    dp, ld_d = _rows(dy, "dy", M, N, dy.dtype, dev)
    xp, ld_x = _rows(x, "x", M, Kd, dy.dtype, dev)
    rc = load().moe_grouped_mm_wgrad(dp, ld_d, xp, ld_x, start, psum, dt, E, N, Kd, M,
                                     _whole(out, "out", (E, N, Kd), out.dtype, dev), TYPE_CODE[out.dtype],
                                     int(accumulate), _word(status, "status", dev), _stream(stream, dev))
    check(rc, "moe_grouped_mm_wgrad")
    return out


def swiglu(gu: torch.Tensor, lay, row_w: Optional[torch.Tensor] = None,
           out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out[r] = silu(g) * u * row_w[r] for the rows r < total of gu = [g | u]
    (row_w None: 1)."""
    dt, dev = _code16(gu, "gu"), _device(gu, "gu")
    M, two = gu.shape
    if two % 2:
        raise ValueError("gu must have an even number of columns")
    if out is None:
        out = _new(torch.zeros, (M, two // 2), gu.dtype, gu, stream)
    gp, ld_g = _rows(gu, "gu", M, two, gu.dtype, dev)
    op, ld_o = _rows(out, "out", M, two // 2, gu.dtype, dev)
    rc = load().moe_swiglu(gp, ld_g, dt, two // 2, _whole(row_w, "row_w", (M,), torch.float32, dev),
                           _word(lay.total, "lay.total", dev), M, op, ld_o, _stream(stream, dev))
    check(rc, "moe_swiglu")
    return out


def swiglu_backward(dh: torch.Tensor, gu: torch.Tensor, lay, row_w: Optional[torch.Tensor] = None,
                    dgu: Optional[torch.Tensor] = None, drow_w: Optional[torch.Tensor] = None,
                    stream=None):
    """(dgu, drow_w): the gradients of swiglu's gu and row_w. ``dgu`` may be
    ``gu`` itself, which is then overwritten."""
    dt, dev = _code16(gu, "gu"), _device(gu, "gu")
    M, two = gu.shape
    if two % 2:
        raise ValueError("gu must have an even number of columns")
    if dgu is None:
        dgu = _new(torch.zeros, (M, two), gu.dtype, gu, stream)
    if drow_w is None:
        drow_w = _new(torch.zeros, (M,), torch.float32, gu, stream)
    gp, ld_g = _rows(gu, "gu", M, two, gu.dtype, dev)
    hp, ld_h = _rows(dh, "dh", M, two // 2, gu.dtype, dev)
    op, ld_o = _rows(dgu, "dgu", M, two, gu.dtype, dev)
    rc = load().moe_swiglu_backward(
        hp, ld_h, gp, ld_g, dt, two // 2, _whole(row_w, "row_w", (M,), torch.float32, dev),
        _word(lay.total, "lay.total", dev), M, op, ld_o, _whole(drow_w, "drow_w", (M,), torch.float32, dev),
        _stream(stream, dev))
    check(rc, "moe_swiglu_backward")
    return dgu, drow_w


# moe_adamw_tensor of include/moe_expand.h
_ADAMW_TENSOR = np.dtype([("p", np.uint64), ("g", np.uint64), ("copy", np.uint64), ("m", np.uint64),
                          ("v", np.uint64), ("m_scale", np.uint64), ("v_scale", np.uint64),
                          ("n", np.int64), ("p_type", np.int32), ("g_type", np.int32),
                          ("copy_type", np.int32), ("reserved", np.int32)])


class AdamW:
    """AdamW (decoupled weight decay) over a list of tensors, one launch per
    step and 400 tensors.

    params   contiguous float32, bfloat16 or float16 tensors on one GPU, updated
             in place
    copies   optional tensors of the same sizes that get the new parameters in
             their own type (the 16-bit weights the products read, beside
             float32 parameters); an entry may be None
    state_bits 32: the moments in float32 (exp_avg, exp_avg_sq). 8: exp_avg and
             the root of exp_avg_sq as e4m3 codes (uint8) with a float32 scale
             per 128 values (exp_avg_scale, exp_avg_sq_scale): 2.06 bytes a
             value instead of 8. A code is 6 to 12 % from the next, so each step
             rounds it at random with an exact mean (repeatably: by the step's
             number and the value's place) once the newest gradient is under
             1/24 of the average (betas[1] over 0.958, after 24 steps); before,
             to nearest. The root then follows its average with a deviation of
             about 15 %; roots under 4e-6 of their block's largest are held at
             that.
    exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale, step: states to go on
             from (a checkpoint's); zeros by default. They are the optimizer's
             from then on.

    step(grads) takes one float32, bfloat16 or float16 gradient per parameter,
    and optionally ``grad_scale``, a float32 device word they are multiplied
    by (a clipping factor, say) without a host read. A step is one of its own
    (its number and lr go with the launch), so it cannot be captured into a CUDA
    graph: capture the forward and backward, and step between the replays.
    """

    def __init__(self, params: Sequence[torch.Tensor], *, lr: float = 1e-3, betas=(0.9, 0.999),
                 eps: float = 1e-8, weight_decay: float = 1e-2, state_bits: int = 32,
                 copies: Optional[Sequence[Optional[torch.Tensor]]] = None,
                 exp_avg: Optional[Sequence[torch.Tensor]] = None,
                 exp_avg_sq: Optional[Sequence[torch.Tensor]] = None,
                 exp_avg_scale: Optional[Sequence[torch.Tensor]] = None,
                 exp_avg_sq_scale: Optional[Sequence[torch.Tensor]] = None, step: int = 0):
        if state_bits not in (32, 8):
            raise ValueError(f"state_bits must be 32 or 8, got {state_bits}")
        if step < 0:
            raise ValueError("step must be >= 0")
        self.lr, self.betas, self.eps, self.weight_decay = lr, tuple(betas), eps, weight_decay
        self.state_bits = state_bits
        self.steps = step
        self.params: List[torch.Tensor] = list(params)
        n = len(self.params)
        self.copies = [None] * n if copies is None else list(copies)
        if len(self.copies) != n:
            raise ValueError(f"{len(self.copies)} copies for {n} parameters")
        for codes, scales, name in ((exp_avg, exp_avg_scale, "exp_avg"),
                                    (exp_avg_sq, exp_avg_sq_scale, "exp_avg_sq")):
            if state_bits == 8 and (codes is None) != (scales is None):
                raise ValueError(f"8-bit {name} and {name}_scale come together: codes without their scales "
                                 "stand for nothing")
        code = torch.float32 if state_bits == 32 else torch.uint8

        def state(given, name, dtype, count):
            if given is None:
                return tuple(torch.zeros(count(p), dtype=dtype, device=p.device) for p in self.params)
            given = tuple(given)
            if len(given) != n:
                raise ValueError(f"{len(given)} tensors in {name} for {n} parameters")
            for i, (s, p) in enumerate(zip(given, self.params)):
                if s.dtype is not dtype or s.numel() != count(p) or not s.is_contiguous() \
                        or s.device != p.device:
                    raise ValueError(f"{name}[{i}] must be contiguous {dtype} with {count(p)} values "
                                     "on the parameter's device")
            return given

        for i, p in enumerate(self.params):
            if p.dtype not in TYPE_CODE or not p.is_contiguous() or not p.is_cuda:
                raise ValueError(f"params[{i}] must be a contiguous float32, bfloat16 or float16 GPU tensor")
            if p.get_device() != self.params[0].get_device():
                raise ValueError(f"params[{i}] is on GPU {p.get_device()}, params[0] on "
                                 f"{self.params[0].get_device()}: an optimizer for each GPU, since a step is "
                                 "one launch")
            c = self.copies[i]
            if c is not None and (c.dtype not in TYPE_CODE or c.numel() != p.numel()
                                  or not c.is_contiguous() or c.device != p.device):
                raise ValueError(f"copies[{i}] must be a contiguous tensor of the parameter's size and device")
        whole = lambda p: p.numel()  # noqa: E731
        self.exp_avg = state(exp_avg, "exp_avg", code, whole)
        self.exp_avg_sq = state(exp_avg_sq, "exp_avg_sq", code, whole)
        if state_bits == 8:
            blocks = lambda p: (p.numel() + STATE_BLOCK - 1) // STATE_BLOCK  # noqa: E731
            self.exp_avg_scale = state(exp_avg_scale, "exp_avg_scale", torch.float32, blocks)
            self.exp_avg_sq_scale = state(exp_avg_sq_scale, "exp_avg_sq_scale", torch.float32, blocks)
        else:
            if exp_avg_scale is not None or exp_avg_sq_scale is not None:
                raise ValueError("scales belong to 8-bit states")
            self.exp_avg_scale = self.exp_avg_sq_scale = ()
        self._table = np.zeros(n, dtype=_ADAMW_TENSOR)
        self._sizes = [p.numel() for p in self.params]
        self._table["n"] = self._sizes
        self._table["m"] = [t.data_ptr() for t in self.exp_avg]
        self._table["v"] = [t.data_ptr() for t in self.exp_avg_sq]
        if state_bits == 8:
            self._table["m_scale"] = [t.data_ptr() for t in self.exp_avg_scale]
            self._table["v_scale"] = [t.data_ptr() for t in self.exp_avg_sq_scale]
        self._devices = [p.get_device() for p in self.params]
        self._types = [p.dtype for p in self.params], [None if c is None else c.dtype for c in self.copies]
        self._table["p_type"] = [TYPE_CODE[t] for t in self._types[0]]
        self._table["copy_type"] = [0 if t is None else TYPE_CODE[t] for t in self._types[1]]
        self._where = None   # (parameters', copies') addresses in the table

    def _locate(self, where) -> None:
        for name, tensors, types in (("parameter", self.params, self._types[0]),
                                     ("copy", self.copies, self._types[1])):
            for i, (t, n, ty, d) in enumerate(zip(tensors, self._sizes, types, self._devices)):
                if t is not None and (t.numel() != n or t.dtype is not ty or not t.is_contiguous()
                                      or t.get_device() != d):
                    raise ValueError(f"{name} {i} has changed its size, type, layout or device since "
                                     "this optimizer was made")
        self._table["p"], self._table["copy"] = where
        self._where = where

    def step(self, grads: Sequence[torch.Tensor], *, grad_scale: Optional[torch.Tensor] = None,
             lr: Optional[float] = None, stream=None) -> None:
        if len(grads) != len(self.params):
            raise ValueError(f"{len(grads)} gradients for {len(self.params)} parameters")
        if not self.params:
            self.steps += 1
            return
        dev = _device(self.params[0], "params[0]")
        # Every gradient is checked at every step; parameters and copies are
        # looked up anew, and checked when they have been given other storage.
        table, sizes, T = self._table, self._sizes, torch.Tensor
        types = [g.dtype for g in grads]
        if list(map(T.numel, grads)) != sizes or not all(map(T.is_contiguous, grads)) \
                or list(map(T.get_device, grads)) != self._devices or not set(types) <= TYPE_CODE.keys():
            raise ValueError("every gradient must be a contiguous float32, bfloat16 or float16 tensor of "
                             "its parameter's size on its device")
        where = list(map(T.data_ptr, self.params)), [0 if c is None else c.data_ptr() for c in self.copies]
        if where != self._where:
            self._locate(where)
        table["g"] = list(map(T.data_ptr, grads))
        table["g_type"] = TYPE_CODE[types[0]] if len(set(types)) == 1 else [TYPE_CODE[t] for t in types]
        if grad_scale is not None and (grad_scale.dtype is not torch.float32 or grad_scale.numel() != 1
                                       or grad_scale.get_device() != dev):
            raise ValueError(f"grad_scale must be a float32 tensor of one element on GPU {dev}")
        rc = load().moe_adamw_step(table.ctypes.data, len(self.params), self.state_bits,
                                   self.lr if lr is None else lr, self.betas[0], self.betas[1],
                                   self.eps, self.weight_decay, self.steps + 1,
                                   None if grad_scale is None else grad_scale.data_ptr(),
                                   _stream(stream, dev))
        check(rc, "moe_adamw_step")
        self.steps += 1


class TrainableExperts:
    """The experts of an expanded-layout MoE layer in bfloat16, with their
    backward pass, for up to ``max_tokens`` tokens; every buffer allocated once.

        forward(x, topk_ids, topk_w, n_valid) -> y [T, H]
        backward(dy) -> (dx [T, H], dtopk_w [T, K]); dw13, dw2 hold the weights'
                        gradients (float32; ``accumulate`` adds to them)
        parameters / gradients: [w13, w2] and [dw13, dw2], for AdamW

    y[t] = sum_k w[t, k] * w2[e] (silu(g) * u), [g | u] = w13[e] x[t], e =
    topk_ids[t, k]. x and topk_ids, topk_w as in ExpandedMoELayer, with x in
    bfloat16; rows t >= n_valid are neither read nor written. backward belongs
    to the last forward, of which the layer keeps what it needs (n_valid and x
    may be refilled before it), and overwrites what that kept of gate_up.
    """

    def __init__(self, w13: torch.Tensor, w2: torch.Tensor, *, K: int, max_tokens: int,
                 align: int = 1):
        from . import Layout, expanded_capacity, workspace_size
        E, twoI, H = w13.shape
        if twoI % 2 or w2.shape != (E, H, twoI // 2):
            raise ValueError("w13 must be [E, 2I, H] and w2 [E, H, I]")
        for name, w in (("w13", w13), ("w2", w2)):
            if w.dtype is not torch.bfloat16 or not w.is_contiguous() or not w.is_cuda:
                raise ValueError(f"{name} must be a contiguous bfloat16 GPU tensor")
        if w2.get_device() != w13.get_device():
            raise ValueError("w13 and w2 must be on the same GPU")
        self.w13, self.w2 = w13, w2
        self.E, self.H, self.I, self.K, self.align, self.T = E, H, twoI // 2, K, align, max_tokens
        dev = w13.device
        M = self.M_cap = max(1, expanded_capacity(max_tokens, K, E, align))
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=dev)  # noqa: E731
        b16 = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=dev)  # noqa: E731
        f32 = lambda *s: torch.zeros(*s, dtype=torch.float32, device=dev)  # noqa: E731
        self.ws = torch.zeros(workspace_size(max_tokens, K, E), dtype=torch.uint8, device=dev)
        self.status = i32(1)
        self.lay = Layout(psum=i32(E), start=i32(E), total=i32(1), m_indices=i32(M),
                          src2dst=i32(max_tokens, K), tile_prefix=i32(E + 1), E=E, align=align, M_cap=M)
        self.xe, self.row_w, self.gu = b16(M, H), f32(M), b16(M, twoI)
        self.h, self.down = b16(M, self.I), b16(M, H)
        self.dh, self.drow_w = b16(M, self.I), f32(M)
        self.y, self.dx, self.dtopk_w = b16(max_tokens, H), b16(max_tokens, H), f32(max_tokens, K)
        self.dw13, self.dw2 = f32(E, twoI, H), f32(E, H, self.I)
        self._n_valid = None          # the last forward's: None or the copy of its word
        self._n_valid_word = i32(1)
        self._ready = False

    @property
    def parameters(self) -> list:
        return [self.w13, self.w2]

    @property
    def gradients(self) -> list:
        return [self.dw13, self.dw2]

    def forward(self, x, topk_ids, topk_w, n_valid=None, stream=None) -> torch.Tensor:
        from . import combine, expand_layout
        dev = _device(self.w13, "w13")
        _rows(x, "x", self.T, self.H, torch.bfloat16, dev)
        _whole(topk_ids, "topk_ids", (self.T, self.K), torch.int32, dev)
        if _whole(topk_w, "topk_w", (self.T, self.K), torch.float32, dev) is None:
            raise ValueError("topk_w is needed")
        _word(n_valid, "n_valid", dev)
        _stream(stream, dev)
        lay = self.lay
        self._ready = False   # from here on the buffers are another forward's
        if n_valid is not None:
            with torch.cuda.stream(stream):
                n_valid = self._n_valid_word.copy_(n_valid.as_strided((1,), (1,)))
        self._n_valid = n_valid
        expand_layout(topk_ids, self.E, self.align, self.M_cap, n_valid, self.ws, self.status, lay,
                      stream)
        expand_rows(x, lay, topk_w, n_valid, self.xe, self.row_w, self.status, stream)
        grouped_matmul(self.xe, self.w13, lay, self.gu, self.status, stream)
        swiglu(self.gu, lay, self.row_w, self.h, stream)
        grouped_matmul(self.h, self.w2, lay, self.down, self.status, stream)
        combine(self.down, lay.src2dst, None, n_valid, self.y, stream)
        self._ready = True
        return self.y

    def backward(self, dy: torch.Tensor, accumulate: bool = False, stream=None):
        from . import combine
        if not self._ready:
            raise RuntimeError("backward needs a forward before it")
        lay, nv, st = self.lay, self._n_valid, self.status
        ddown = expand_rows(dy, lay, None, nv, self.down, None, st, stream)   # a dy it refuses costs nothing
        self._ready = False
        grouped_matmul_wgrad(ddown, self.h, lay, self.dw2, accumulate, status=st, stream=stream)
        grouped_matmul_dgrad(ddown, self.w2, lay, self.dh, st, stream)
        dgu, drow_w = swiglu_backward(self.dh, self.gu, lay, self.row_w, self.gu, self.drow_w, stream)
        grouped_matmul_wgrad(dgu, self.xe, lay, self.dw13, accumulate, status=st, stream=stream)
        dxe = grouped_matmul_dgrad(dgu, self.w13, lay, self.down, st, stream)
        combine(dxe, lay.src2dst, None, nv, self.dx, stream)
        collect_row_grads(drow_w, lay, nv, self.dtopk_w, stream)
        return self.dx, self.dtopk_w
