"""Inputs of the 4-bit product whose sums are exact in fp32, in whatever order:
x of -1, 0 and 1 (an eighth of it not 0), scales of 1/4 to 2. A sum is a multiple of
1/4 and at most Kd 15 2 < 2^22 for Kd <= 65536, which leaves 24 bits enough. So a
result is its exact value, rounded once, and nothing that is lost or misplaced hides
behind a tolerance that grows with the contraction."""
import torch

F64 = torch.float64


def inputs(rows, E, N, Kd, group, dtype, seed):
    """(x [rows, Kd], codes, scales, zero points) on the CPU."""
    g = torch.Generator().manual_seed(seed)
    draw = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g)  # noqa: E731
    x = (draw(0, 8, rows, Kd) == 0) * (2 * draw(0, 2, rows, Kd) - 1)
    codes = draw(0, 256, E, N, Kd // 2).to(torch.uint8)
    scales = 2.0 ** draw(-2, 2, E, N, Kd // group).double()
    zeros = draw(0, 16, E, N, Kd // group).to(torch.uint8)
    return x.to(dtype), codes, scales.to(dtype), zeros


def dense(codes, scales, zeros):
    """One expert's weights [N, Kd] in 64 bits."""
    q = torch.stack([codes & 15, codes >> 4], dim=2).flatten(1).to(F64)
    group = q.shape[1] // scales.shape[1]
    wide = lambda t: t.to(F64).repeat_interleave(group, 1)  # noqa: E731
    return (q - wide(zeros)) * wide(scales)
