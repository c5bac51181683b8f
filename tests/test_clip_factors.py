"""lora_clip_gradients where the factor is far below what float32 holds.

Tolerances are those of test_clip.py (a factor of any size is a float32 number times a
power of two, which adds no rounding but a subnormal result's).
"""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(__file__))
from test_clip import compare, run  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("power", [127, 90, 60, 0])
def test_factors_of_any_size(dtype, power):
    g = torch.Generator().manual_seed(power)
    t = [(torch.rand(5000, generator=g, dtype=torch.float64) * 2.0 ** power).to(dtype), torch.full((3,), 2.0 ** power, dtype=dtype)]
    for limit in (2.0 ** -40, 2.0 ** -59, 2.0 ** -61, 2.0 ** -75, 1e-30, 2.0 ** -110, 1e-40, 2.0 ** -140):
        got, out, _ = run(t, 1, limit)
        compare(t, got, out, 1, limit)
