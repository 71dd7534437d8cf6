"""The exact inputs of the 4-bit product's tests show what a kernel could get wrong
over a long contraction: each mistake, planted in the definition, changes nearly every
rounded result."""
import pytest
import torch

from w4_exact_inputs import F64, dense, inputs

N, ROWS = 40, 4


def shifted(t, last):
    """The last columns of t one to the left."""
    out = t.clone()
    out[:, -last:] = t[:, -last - 1:-1]
    return out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("Kd,group", [(65536, 32), (16384, 64), (16384, 128)])
def test_mistakes_show(Kd, group, dtype):
    x, codes, scales, zeros = (t[0] if t.dim() == 3 else t for t in inputs(ROWS, 1, N, Kd, group, dtype, Kd))
    x = x.to(F64)
    w = dense(codes, scales, zeros)
    exact = x @ w.T
    want = exact.to(dtype)
    # exact in fp32, and far from fp16's largest value
    assert torch.equal(exact, exact.float().to(F64)) and (exact * 4 == (exact * 4).round()).all()
    assert exact.abs().max() < 2 ** 14 and (x.abs() @ w.abs().T).max() < 2 ** 22

    def lost(a, b):
        keep = torch.ones(Kd, dtype=torch.bool)
        keep[a:b] = False
        return (x * keep) @ w.T

    def with_weights(*a):
        return x @ dense(*a).T

    sixteenth = Kd // group // 16
    mistakes = {
        "first stage lost": lost(0, 128),
        "last stage lost": lost(Kd - 128, Kd),
        "a stage twice": exact + x[:, 1024:1152] @ w[:, 1024:1152].T,
        "an eighth of the contraction lost": lost(Kd // 8, Kd // 4),
        "scales a group behind at the end": with_weights(codes, shifted(scales, sixteenth), zeros),
        "zero points a group behind at the end": with_weights(codes, scales, shifted(zeros, sixteenth)),
        "codes of a byte swapped": with_weights((codes >> 4) | (codes << 4), scales, zeros),
        "zero points left out": with_weights(codes, scales, torch.full_like(zeros, 8)),
        "nothing": torch.zeros_like(exact),
    }
    for name, got in mistakes.items():
        assert (got.to(dtype) != want).double().mean() > 0.75, name


def test_the_sum_of_a_stage_is_seen_in_fp16():
    """16 terms of a stage, against a result of some hundreds in steps of 1/2."""
    x, codes, scales, zeros = inputs(8, 1, N, 65536, 32, torch.float16, 1)
    x, w = x.to(F64), dense(codes[0], scales[0], zeros[0])
    exact = x @ w.T
    for stage in range(0, 512, 37):
        a = stage * 128
        less = exact - x[:, a:a + 128] @ w[:, a:a + 128].T
        assert (less.to(torch.float16) != exact.to(torch.float16)).double().mean() > 0.9, stage
