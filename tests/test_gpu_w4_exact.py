"""The experts' product over 4-bit weights on inputs whose sums are exact: every
result is the formula's, rounded once, with no tolerance."""
import pytest
import torch

from test_gpu_w4 import layout_of, mx  # noqa: F401
from w4_exact_inputs import F64, dense, inputs

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16

# rows of each expert, N, Kd, group
CASES = {
    "few rows": ([1, 0, 2, 8, 1], 200, 7168, 128),
    "few rows, groups of 64": ([1, 0, 2, 8, 1], 200, 6528, 64),
    "few rows, groups of 32": ([3, 1], 72, 4096 + 32, 32),
    "few rows, long": ([1, 4], 72, 32768, 128),
    "more scales than the form for few rows takes": ([1, 3], 40, 65536, 32),
    "a cluster": ([40], 264, 8192, 128),
    "a cluster, groups of 64": ([40], 264, 8192, 64),
    "a cluster, groups of 32": ([40], 264, 8192, 32),
    "a cluster, ragged": ([33, 12], 128, 16384 + 128, 128),
    "a cluster, long": ([20, 0, 70], 72, 65536, 64),
    "a cluster, long, groups of 32": ([20, 0, 70], 72, 65536, 32),
    "whole tiles": ([48, 33, 97, 0, 19, 13], 1160, 2048 + 64, 64),
    "whole tiles, groups of 32": ([16, 33, 0, 17, 30, 9], 1032, 2048 + 32, 32),
    "whole tiles, groups of 128": ([64, 5, 130, 0, 65, 31], 1288, 4096, 128),
}


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("name", CASES)
def test_exact(mx, name, dtype):  # noqa: F811
    counts, N, Kd, group = CASES[name]
    lay, bounds = layout_of(mx, counts, pairs=sum(counts))
    x, codes, scales, zeros = (t.cuda() for t in inputs(lay.M_cap, len(counts), N, Kd, group, dtype, N + Kd))
    out = mx.grouped_matmul_w4(x, codes, scales, lay, zeros=zeros)
    for e, (a, b) in enumerate(bounds):
        exact = x[a:b].to(F64) @ dense(codes[e], scales[e], zeros[e]).T
        assert exact.numel() == 0 or exact.abs().max() < 2 ** 15
        assert torch.equal(out[a:b], exact.to(dtype)), e
