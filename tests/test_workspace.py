"""The workspaces of lora_linear and of the loss: one that is sized for the
largest batch serves every smaller one, whatever it holds."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(__file__))
import test_linear as linear  # noqa: E402
import test_loss as loss  # noqa: E402


def _never_decreases(size, most):
    last = 0
    for n in list(range(0, min(most, 6000))) + list(range(6000, most, 997)):
        now = size(n)
        assert now >= last, "%d tokens need %d bytes, fewer need %d" % (n, now, last)
        last = now


@pytest.mark.parametrize("loras,hidden,widths,rank", [
    (32, 4096, [4096, 1024, 1024], 128), (128, 8192, [8192, 1024, 1024], 64), (4, 72, [4104, 72], 16),
    (1023, 520, [136], 8), (1, 8, [1024], 24)])
@pytest.mark.parametrize("backward", [False, True])
def test_linear_sizes_never_decrease(loras, hidden, widths, rank, backward):
    sgl = linear.lib()
    _never_decreases(lambda n: sgl.lora_linear_workspace_bytes(n, loras, hidden, widths, rank, backward), 70000)


@pytest.mark.parametrize("hidden,vocab", [(4096, 128256), (8192, 32000), (72, 5003), (264, 1 << 20), (8, 300),
                                          (16384, 256), (8, 1 << 24)])
@pytest.mark.parametrize("backward", [False, True])
def test_loss_sizes_never_decrease(hidden, vocab, backward):
    sgl = loss.lib()
    _never_decreases(lambda n: sgl.lora_cross_entropy_workspace_bytes(n, hidden, vocab, backward), 140000)


@pytest.mark.gpu
def test_a_large_batchs_workspace_serves_small_ones():
    """A ragged last batch with the buffers of the full one."""
    sgl = linear.lib()
    for n in (1, 70, 517, 1100):
        c = linear.Case(n=n, hidden=136, widths=[1160, 72], rank=24, loras=5)
        r = linear.Run(c)
        r.workspace = torch.zeros(sgl.lora_linear_workspace_bytes(1100, c.loras, c.hidden, c.widths, c.rank, True),
                                  dtype=torch.uint8, device="cuda")
        r.forward()
        r.backward()
        linear.check(c, r.outputs())
    for n in (1, 40, 300, 1100):
        c = loss.Case(n=n, hidden=72, vocab=5003)
        r = loss.Run(c)
        r.workspace = torch.full((sgl.lora_cross_entropy_workspace_bytes(1100, 72, 5003, True),), 0xff,
                                 dtype=torch.uint8, device="cuda")
        r.forward()
        r.backward()
        loss.check(c, r.outputs())


@pytest.mark.gpu
@pytest.mark.parametrize("n,widths", [(1, [4104, 72]), (70, [4104, 72]), (300, [2056]), (1500, [72])])
def test_what_a_linear_workspace_holds_does_not_matter(n, widths):
    """The same memory serves the loss in between, or holds anything."""
    c = linear.Case(n=n, hidden=72, widths=widths, rank=16, loras=6)
    r = linear.Run(c)
    for held in (0xff, 0x01, None):
        if held is not None:
            r.workspace.fill_(held)
        for t in [r.buf, r.dbuf, r.y, r.dx] + r.da + r.db + r.dbias:
            t.fill_(float("nan"))
        r.forward()
        r.backward()
        linear.check(c, r.outputs())


@pytest.mark.gpu
def test_an_empty_batch_launches_nothing():
    """The status of a call without tokens is not written: the workspace stays as it was."""
    c = loss.Case(n=0, hidden=16, vocab=300)
    r = loss.Run(c)
    before = r.workspace.clone()
    r.forward()
    torch.cuda.synchronize()
    assert torch.equal(r.workspace, before)
