"""lora_clip_gradients where the factor is far below what float32 holds, and where it
is 1: gradients that are not scaled come out bit for bit, NaN and zeros' signs with them.

Tolerances are those of test_clip.py (a factor of any size is a float32 number times a
power of two, which adds no rounding but a subnormal result's).
"""
import math
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(__file__))
from test_clip import compare, run  # noqa: E402
from test_linear import lib  # noqa: E402

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


def bits(t):
    return t.contiguous().view(torch.int16 if t.dtype is BF16 else torch.int32)


def patterns(dtype, n):
    """Every kind of number, among them NaN of both signs with other bits set."""
    if dtype is BF16:
        return (torch.arange(n) * 37 % 65536).to(torch.int32).to(torch.int16).view(BF16)
    g = torch.Generator().manual_seed(1)
    odd = torch.tensor([0x7f800001, 0x7fc12345, -0x7fffff, -0x3fffff, -0x800000, -0x80000000, 1, -0x7fffffff, 0x7f800000])
    v = torch.randint(-2 ** 31, 2 ** 31, (n,), generator=g)
    v[::11] = odd[torch.arange(len(v[::11])) % len(odd)]
    return v.to(torch.int32).view(F32)


@pytest.mark.gpu
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_what_is_not_scaled_keeps_its_bits(dtype, shift):
    sgl = lib()
    groups, each = 3, 70000
    t = torch.randn((groups, each), generator=torch.Generator().manual_seed(5)).to(dtype)
    t[1] = patterns(dtype, each)                   # not finite
    t[2] *= 1e-4                                   # below the limit
    dev = t.cuda()
    flat = torch.full((groups * each + 8,), 9.0, dtype=dtype, device="cuda")
    out = flat[shift:shift + groups * each].view(groups, each)
    norms = torch.empty(groups, device="cuda")
    ws = torch.full((sgl.lora_clip_gradients_workspace_bytes([dev], groups),), 0xFF, dtype=torch.uint8, device="cuda")
    for limit, kept in ((1.0, [1, 2]), (math.inf, [0, 1, 2])):
        flat.fill_(9.0)
        sgl.lora_clip_gradients([dev], norms, limit, ws, out=[out])
        assert torch.equal(bits(dev).cpu(), bits(t))
        assert torch.equal(bits(out).cpu()[kept], bits(t)[kept])
        finite = norms.cpu().isfinite()
        assert finite.tolist() == [True, False, True]
        compare([t[[0, 2]]], norms[[0, 2]], [out[[0, 2]]], 2, limit)
        assert (flat[:shift] == 9.0).all() and (flat[shift + groups * each:] == 9.0).all()
    sgl.lora_clip_gradients([dev], norms, 1.0, ws)
    assert torch.equal(bits(dev).cpu()[1:], bits(t)[1:])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_streamed_results_keep_their_bits(dtype):
    """Gradients of more bytes than the last-level cache, which take other instructions."""
    sgl = lib()
    size = 2 if dtype is BF16 else 4
    each = (224 << 20) // size // 2 + 3
    t = torch.empty((2, each), dtype=dtype, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(2))
    t[1, :100000] = patterns(dtype, 100000).cuda()
    flat = torch.empty(2 * each, dtype=dtype, device="cuda")
    out, norms = flat.view(2, each), torch.empty(2, device="cuda")
    ws = torch.empty(sgl.lora_clip_gradients_workspace_bytes([t], 2), dtype=torch.uint8, device="cuda")
    sgl.lora_clip_gradients([t], norms, 1.0, ws, out=[out])
    assert torch.equal(bits(out[1]), bits(t[1]))
    want = t[0].double().square().sum().sqrt().item()
    assert abs(norms[0].item() - want) <= want * 2.0 ** -23 and not math.isfinite(norms[1].item())
    rel = 2.0 ** -8 + 2.0 ** -22 if dtype is BF16 else 2.0 ** -22
    exact = t[0].double() * (1.0 / (want + 1e-6))
    assert ((out[0].double() - exact).abs() <= exact.abs() * rel + 2.0 ** -133).all()
