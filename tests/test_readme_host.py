"""The README's function that makes 4-bit weights, run as it stands there."""
import os
import re

import pytest
import torch

from expanded_layout_expert_gb300 import w4

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def to_four_bits():
    with open(os.path.join(ROOT, "README.md"), encoding="utf-8") as f:
        text = f.read()
    source = re.search(r"^def to_four_bits\(.*?^```", text, re.S | re.M).group(0)[:-3]
    names = {"torch": torch}
    exec(source, names)
    return names["to_four_bits"]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_weights_in_four_bits(group, dtype):
    """Each weight is off by at most half a step, or by what the largest of a group
    loses: its place is up to 15 (1 + u) and half a step more by the zero point's
    rounding, and 15 is the last one."""
    g = torch.Generator().manual_seed(group)
    w = torch.randn(3, 16, 256, generator=g) * torch.randn(3, 16, 256 // 32, generator=g).exp().repeat_interleave(32, 2)
    w[0, 0] = 0.0
    w[0, 1] = w[0, 1].abs() + 1
    w[0, 2] = -w[0, 2].abs() - 1
    w = w.to(dtype)
    codes, scales, zeros = to_four_bits()(w, group)
    assert w4._weights(codes, scales) == (3, 16, 256, group)
    assert codes.dtype == zeros.dtype == torch.uint8 and scales.dtype == dtype
    assert zeros.shape == scales.shape and zeros.max() <= 15
    q = torch.stack([codes & 15, codes >> 4], dim=3).flatten(2).double()
    wide = lambda t: t.double().repeat_interleave(group, 2)  # noqa: E731
    back = (q - wide(zeros)) * wide(scales)
    most = 0.5 + 15 * torch.finfo(dtype).eps / 2 + 1e-4   # 1e-4: the divisions in fp32
    assert ((back - w.double()).abs() <= most * wide(scales)).all()
    assert (back[0, 0] == 0).all()
