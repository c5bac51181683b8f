"""LoraGradients over tensors that change between calls while their address stays: a
shorter view, another type, another shape or order of the same memory.  A call goes by
the tensors as they are, or refuses them; nothing outside them is read or written.

Tolerances are those of test_clip.py.
"""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(__file__))
from test_clip import compare  # noqa: E402
from test_linear import lib  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


def held(shapes, groups, own_results, dtype=F32):
    sgl = lib()
    g = torch.Generator().manual_seed(len(shapes))
    grads = [torch.randn(s, generator=g).to(dtype).cuda() for s in shapes]
    out = [torch.full_like(t, 9.0) for t in grads] if own_results else None
    h = sgl.LoraGradients(grads, out)
    norms = torch.full((groups,), float("nan"), device="cuda")
    ws = torch.full((sgl.lora_clip_gradients_workspace_bytes(h, groups),), 0xFF, dtype=torch.uint8, device="cuda")
    return grads, out, h, norms, ws


@pytest.mark.gpu
@pytest.mark.parametrize("own_results", [False, True])
def test_shorter_at_the_same_address(own_results):
    sgl = lib()
    grads, out, h, norms, ws = held([(1000,), (3, 40)], 1, own_results)
    whole, whole_out = grads[0].data, out[0].data if own_results else grads[0].data
    tail = whole_out[300:].clone()
    grads[0].data = whole[:300]
    if own_results:
        out[0].data = whole_out[:300]
    given = [t.cpu().clone() for t in grads]
    sgl.lora_clip_gradients(h, norms, 1.0, ws)
    compare(given, norms, out if own_results else grads, 1, 1.0)
    assert torch.equal(whole_out[300:], tail)
    # and the whole again
    grads[0].data = whole
    if own_results:
        out[0].data = whole_out
    given = [t.cpu().clone() for t in grads]
    sgl.lora_clip_gradients(h, norms, 0.5, ws)
    compare(given, norms, out if own_results else grads, 1, 0.5)


@pytest.mark.gpu
def test_another_type_at_the_same_address():
    sgl = lib()
    grads, _, h, norms, ws = held([(1000,), (3, 40)], 1, False)
    whole = grads[0].data
    whole.view(BF16)[:1000].copy_(torch.randn(1000, generator=torch.Generator().manual_seed(3)))
    tail = whole[500:].clone()
    grads[0].data = whole.view(BF16)[:1000]          # as many numbers, of half the size
    given = [t.cpu().clone() for t in grads]
    sgl.lora_clip_gradients(h, norms, 1.0, ws)
    compare(given, norms, grads, 1, 1.0)
    assert torch.equal(whole[500:], tail)
    grads[0].data = whole.view(torch.float16)[:1000]
    before = whole.clone()
    with pytest.raises(TypeError):
        sgl.lora_clip_gradients(h, norms, 0.1, ws)
    assert torch.equal(whole, before)


@pytest.mark.gpu
@pytest.mark.parametrize("own_results", [False, True])
def test_another_order_or_shape_at_the_same_address(own_results):
    sgl = lib()
    grads, out, h, norms, ws = held([(6, 8), (6, 100)], 6, own_results)
    to = out if own_results else grads
    keep, before = to[0].data, [t.clone() for t in grads]
    for bad in (keep.t(), keep.as_strided((6, 8), (1, 6)), keep.as_strided((6, 4), (8, 1)), keep.view(8, 6),
                keep.view(48), keep[:3]):
        to[0].data = bad
        with pytest.raises(sgl.LoraError):
            sgl.lora_clip_gradients(h, norms, 1e-3, ws)
    to[0].data = keep
    assert all(torch.equal(a, b) for a, b in zip(grads, before))
    given = [t.cpu().clone() for t in grads]
    sgl.lora_clip_gradients(h, norms, 1.0, ws)
    compare(given, norms, to, 6, 1.0)


@pytest.mark.gpu
def test_refused_tensors_leave_the_list_as_it_was():
    """A call that refuses changed tensors keeps nothing of them: with the old tensors
    back, the next call is that of the old ones."""
    sgl = lib()
    grads, _, h, norms, ws = held([(5, 30), (5, 7)], 5, False)
    keep = grads[1].data
    for bad in (keep.half(), keep[:, ::2], keep[:4], torch.zeros((4, 7), device="cuda")):
        grads[1].data = bad
        with pytest.raises((TypeError, sgl.LoraError)):
            sgl.lora_clip_gradients(h, norms, 1.0, ws)
    grads[1].data = keep
    given = [t.cpu().clone() for t in grads]
    sgl.lora_clip_gradients(h, norms, 1.0, ws)
    compare(given, norms, grads, 5, 1.0)
