"""Values that comparisons after nan_to_num would let pass: infinities and NaN out of
lora_mx_dequantize, and a whole step's outputs, eager and replayed, bit for bit.
"""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(__file__))
import test_mx  # noqa: E402
import test_mx_step  # noqa: E402
from test_linear import lib  # noqa: E402


def same(got, want):
    """Equal values, NaN in the same places."""
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(got[~nan], want[~nan])


@pytest.mark.gpu
@pytest.mark.parametrize("to", [torch.bfloat16, torch.float32])
def test_every_code_and_scale(to):
    sgl = lib()
    codes = (torch.arange(256 * 16) % 256).reshape(256, 16).to(torch.uint8)
    scales = torch.full((256, 4), 255, dtype=torch.uint8)
    scales[:, 0] = torch.arange(256)
    out = torch.empty((256, 32), dtype=to, device="cuda")
    sgl.lora_mx_dequantize(codes.cuda(), scales.cuda(), out)
    both = torch.stack((codes & 15, codes >> 4), 2).flatten(1).long()
    value = torch.cat((test_mx.GRID, -test_mx.GRID))[both] * torch.exp2(torch.arange(256).double() - 127)[:, None]
    value[255] = float("nan")
    want = value.to(to)
    assert torch.isinf(want).any() and torch.isnan(want[255]).all() and not torch.isnan(want[:255]).any()
    same(out.cpu(), want)
    assert torch.equal(torch.signbit(out.cpu())[:255], torch.signbit(want)[:255])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["normal", "rows", "borders", "tiny", "zeros", "not finite", "largest"])
def test_there_and_back(dtype, kind):
    sgl = lib()
    n, k = 37, 1048
    x = test_mx.numbers(kind, n, k, 3, dtype)
    held = test_mx.quantized(x.double())[2]
    code_bytes, scale_bytes = sgl.lora_mx_row_bytes(k)
    codes = torch.empty((n, code_bytes), dtype=torch.uint8, device="cuda")
    scales = torch.empty((n, scale_bytes), dtype=torch.uint8, device="cuda")
    sgl.lora_mx_quantize(x.cuda(), codes, scales)
    for to in (torch.bfloat16, torch.float32):
        out = torch.empty((n, k), dtype=to, device="cuda")
        sgl.lora_mx_dequantize(codes, scales, out)
        same(out.cpu(), held.to(to))


@pytest.mark.gpu
@pytest.mark.parametrize("acts,n", [("bf16", 20), ("bf16", 70), ("mxfp4", 20), ("mxfp4", 300)])
def test_step_has_the_same_bits_eager_and_replayed(acts, n):
    """(K is too short here for a shrink that adds its parts in no order.)"""
    step = test_mx_step.Step(acts, n, hidden=136, widths=[72, 64], rank=24, loras=5, vocab=203, seed=n + 1)
    outputs = lambda: [step.y, step.loss, step.lse, step.dy, step.dx, step.norms] + step.grads + step.out
    step.run()
    step.check()
    first = [t.clone() for t in outputs()]
    step.run()
    assert all(torch.equal(a, b) for a, b in zip(first, outputs()))
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step.run()
    for k in range(3):
        for t in outputs():
            t.fill_(float("nan"))
        step.workspace.fill_(0x55 * k)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, outputs()))
