"""lora_linear_mx over rows that are far apart, and over batches that follow others.

Codes and scales, and the activations, at the largest distances that the calls take
and just past those at which they change their kernel: offsets within a tile near
2^32 bytes.  Tolerances are those of test_mx.py; the memory between the rows is never
read (the buffers are not initialised).
"""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(__file__))
import test_mx  # noqa: E402
from test_linear import lib  # noqa: E402

FAR = 1 << 25      # the largest distance of two rows of codes, bytes


def apart(t, pitch):
    """t's rows `pitch` elements apart in memory of their own."""
    flat = torch.empty((t.shape[0] - 1) * pitch + t.shape[1], dtype=t.dtype, device="cuda")
    out = flat.as_strided(t.shape, (pitch, 1))
    out.copy_(t)
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("acts,n,widths", [
    ("bf16", 20, [72]), ("mxfp4", 20, [72]),          # few tokens
    ("bf16", 40, [136]), ("mxfp4", 40, [136]),        # 64 x 64 tiles, from the codes and of them
    ("bf16", 15000, [136]), ("mxfp4", 15000, [136])])  # 128 x 128 tiles: 127 rows of codes apart
def test_codes_far_apart(acts, n, widths):
    c = test_mx.MxCase(acts=acts, n=n, hidden=72, widths=widths, rank=8, loras=3)
    r = test_mx.MxRun(c)
    r.codes = apart(r.codes, FAR)
    r.forward()
    r.backward()
    test_mx.check(c, r.outputs())


@pytest.mark.gpu
@pytest.mark.parametrize("acts", ["bf16", "mxfp4"])
@pytest.mark.parametrize("n", [20, 40])
def test_scales_far_apart(acts, n):
    c = test_mx.MxCase(acts=acts, n=n, hidden=168, widths=[136], rank=8, loras=3)
    r = test_mx.MxRun(c)
    r.scales = apart(r.scales, FAR + 4)
    r.forward()
    r.backward()
    test_mx.check(c, r.outputs())


@pytest.mark.gpu
@pytest.mark.parametrize("acts", ["bf16", "mxfp4"])
@pytest.mark.parametrize("n,over", [(20, 0), (300, 0), (300, 8)])
def test_activations_far_apart(acts, n, over):
    """Rows that end just below and just above 2^32 bytes."""
    c = test_mx.MxCase(acts=acts, n=n, hidden=136, widths=[72], rank=8, loras=3)
    r = test_mx.MxRun(c)
    pitch = ((1 << 32) - 1) // (2 * n) // 8 * 8 + over
    assert (2 * n * pitch >= 1 << 32) == (over > 0)
    r.x = apart(r.x, pitch)
    r.forward()
    r.backward()
    test_mx.check(c, r.outputs())


@pytest.mark.gpu
@pytest.mark.parametrize("acts", ["bf16", "mxfp4"])
@pytest.mark.parametrize("n,widths,loras", [(1, [72, 40], 3), (20, [72, 40], 3), (200, [72, 40], 3), (200, [72], 90),
                                            (520, [6144, 8], 5), (2050, [5400, 72], 5)])
def test_ids_out_of_range_and_batches_without_adapters(acts, n, widths, loras):
    """Ids out of range count as none, with biases; a batch of none follows in the same
    metadata, whose order and ids are those of the batch before, and then the first again."""
    sgl = lib()
    c = test_mx.MxCase(acts=acts, n=n, hidden=72, widths=widths, rank=8, loras=loras)
    wild = torch.tensor([loras, loras + 1, -2, 2 ** 31 - 1, -2 ** 31, 1 << 20], dtype=torch.int64)
    given = c.ids.long()
    given[::7] = wild[torch.arange(len(given[::7])) % len(wild)]
    known = torch.where((given >= 0) & (given < loras), given, torch.full_like(given, -1)).to(torch.int32)
    none = torch.full((n,), -1, dtype=torch.int32)
    r = test_mx.MxRun(c)
    for ids, of in ((given.to(torch.int32), known), (none, none), (given.to(torch.int32), known)):
        sgl.lora_prepare_meta(ids.cuda(), r.meta)
        for t in [r.buf, r.dbuf, r.y, r.dx] + r.da + r.db + r.dbias:
            t.fill_(float("nan"))
        r.workspace.fill_(0xFF)
        r.forward()
        r.backward()
        c.ids = of
        test_mx.check(c, r.outputs())
