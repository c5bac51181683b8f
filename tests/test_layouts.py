"""Rows further apart than their length, columns before and after the slices, and
ids out of range, on every tile of lora_linear, the loss and their backward
passes."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(__file__))
import test_linear as linear  # noqa: E402
import test_loss as loss  # noqa: E402

LINEAR = {   # (case, results that the tile in question makes)
    "few tokens": (dict(n=20, hidden=264, widths=[136, 40], rank=24, loras=5), ("y", "dx", "s", "u", "da", "db", "dbias")),
    "64 x 64": (dict(n=200, hidden=136, widths=[72, 40], rank=40, loras=3), ("y", "dx", "s", "u", "da", "db", "dbias")),
    "64 x 64 in two rounds, y": (dict(n=129, hidden=72, widths=[12800, 8], rank=40, loras=7), ("y", "s")),
    "64 x 64 in two rounds, dx": (dict(n=129, hidden=12808, widths=[40, 24], rank=16, loras=7), ("dx", "u", "da", "db", "dbias")),
    "128 x 128, y": (dict(n=520, hidden=136, widths=[8000, 200], rank=16, loras=5), ("y", "s")),
    "128 x 128, dx": (dict(n=520, hidden=8200, widths=[72, 64], rank=72, loras=5), ("dx", "u", "da", "db", "dbias")),
    "256 x 256, y": (dict(n=2050, hidden=200, widths=[5400, 72], rank=24, loras=9), ("y", "s")),
    "256 x 256, y, ranks up to 16": (dict(n=2050, hidden=200, widths=[5400, 72], rank=8, loras=90), ("y", "s")),
    "256 x 256, y, many slices": (dict(n=2050, hidden=136, widths=[8, 16, 24, 5000, 40, 8, 16, 400], rank=128, loras=30),
                                  ("y", "s")),
    "256 x 256, dx, ranks up to 16": (dict(n=2050, hidden=5400, widths=[72, 40], rank=16, loras=90), ("dx", "u")),
    "256 x 256, dx, many slices": (dict(n=2050, hidden=5400, widths=[8, 16, 24, 72], rank=128, loras=30), ("dx", "u")),
    "256 x 256, dx": (dict(n=2050, hidden=5400, widths=[136, 72], rank=40, loras=9), ("dx", "u", "da", "db", "dbias")),
}


@pytest.mark.gpu
@pytest.mark.parametrize("stride,offset,extra", [(8, 24, 40), (72, 0, 8), (0, 8, 0)])
@pytest.mark.parametrize("name", list(LINEAR))
def test_linear(name, stride, offset, extra):
    kw, keys = LINEAR[name]
    c = linear.Case(**kw, stride=stride, offset=offset, extra=extra)
    r = linear.Run(c)
    r.forward()
    r.backward()
    linear.check(c, r.outputs(), keys)
    if stride:     # nothing is written between the rows
        for t in (r.y, r.dx):
            wide = t.as_strided((t.shape[0], t.stride(0)), (t.stride(0), 1))
            assert torch.isnan(wide[:, t.shape[1]:]).all()


LOSS = {
    "128 x 32": dict(n=20, hidden=264, vocab=3001),
    "64 x 64": dict(n=130, hidden=72, vocab=1003),
    "128 x 128": dict(n=200, hidden=520, vocab=25001),
    "256 x 256": dict(n=600, hidden=1032, vocab=16600),
}


@pytest.mark.gpu
@pytest.mark.parametrize("stride", [8, 72])
@pytest.mark.parametrize("name", list(LOSS))
def test_loss(name, stride):
    c = loss.Case(**LOSS[name], stride=stride)
    r = loss.Run(c)
    r.forward()
    r.backward()
    loss.check(c, r.outputs())
    for t in (r.dx, r.dw):
        wide = t.as_strided((t.shape[0], t.stride(0)), (t.stride(0), 1))
        assert torch.isnan(wide[:, t.shape[1]:]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("n,widths,loras", [(20, [72, 40], 3), (200, [72, 40], 3), (200, [72], 90), (2050, [5400, 72], 5)])
def test_ids_out_of_range_with_biases(n, widths, loras):
    """They count as none: no adapter, no bias of an adapter, no gradient."""
    c = linear.Case(n=n, hidden=72, widths=widths, rank=8, loras=loras)
    wild = torch.tensor([loras, loras + 1, -2, 2 ** 31 - 1, -2 ** 31, 1 << 20], dtype=torch.int64)
    given = c.ids.long()
    given[::7] = wild[torch.arange(len(given[::7])) % len(wild)]
    c.ids = given.to(torch.int32)
    r = linear.Run(c)
    r.forward()
    r.backward()
    got = r.outputs()
    assert int(r.meta.views()["status"].item()) == linear.lib().LORA_ERR_ID_RANGE
    c.ids = torch.where((given >= 0) & (given < loras), given, torch.full_like(given, -1)).to(torch.int32)
    linear.check(c, got)


@pytest.mark.gpu
@pytest.mark.parametrize("n,loras", [(1, 3), (20, 4), (64, 12), (300, 6), (2000, 300)])
def test_batches_prepared_with_their_first_layer(n, loras):
    """lora_prepare_shrink_expand writes the batch's metadata in its own launch (by
    id, or sorted by every workgroup); lora_linear and its backward pass go by it."""
    sgl = linear.lib()
    c = linear.Case(n=n, hidden=136, widths=[72, 40], rank=16, loras=loras)
    r = linear.Run(c)
    r.meta = sgl.LoraMeta(c.loras, c.n)
    y = torch.zeros(n, sum(c.widths), dtype=torch.bfloat16, device="cuda")
    first = torch.empty_like(r.buf)
    sgl.lora_prepare_shrink_expand(c.ids.cuda(), r.x, r.a, r.b, None, first, y, r.meta, c.scale)
    r.forward()
    r.backward()
    linear.check(c, r.outputs())
