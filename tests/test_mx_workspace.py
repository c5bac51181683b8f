"""The workspace of lora_linear_mx: room for the matrix where a batch of so many tokens
may need it, none for the forward pass of a few tokens, and nothing written behind it.

Tolerances are those of test_mx.py.
"""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(__file__))
import test_mx  # noqa: E402
from test_linear import lib  # noqa: E402


def test_few_tokens_need_no_room_for_the_matrix():
    sgl = lib()
    hidden, out, widths, rank = 4096, 6144, [4096, 1024, 1024], 16
    mx = lambda n, backward: sgl.lora_linear_mx_workspace_bytes(n, 32, hidden, out, widths, rank, backward)
    linear = lambda n, backward: sgl.lora_linear_workspace_bytes(n, 32, hidden, widths, rank, backward)
    for n in (0, 1, 16, 32):
        assert mx(n, False) == linear(n, False)
        assert mx(n, True) >= linear(n, True) + 2 * out * hidden
    assert mx(33, False) >= linear(33, False) + 2 * out * hidden
    sizes = [mx(n, False) for n in range(0, 100)]
    assert sizes == sorted(sizes)


@pytest.mark.gpu
@pytest.mark.parametrize("acts", ["bf16", "mxfp4"])
@pytest.mark.parametrize("n", [1, 16, 17, 32, 33, 200, 1100])
def test_nothing_is_written_behind_it(acts, n):
    sgl = lib()
    c = test_mx.MxCase(acts=acts, n=n, hidden=264, widths=[136, 2400], rank=24, loras=5)
    for backward in (False, True):
        r = test_mx.MxRun(c)
        nbytes = sgl.lora_linear_mx_workspace_bytes(n, c.loras, c.hidden, c.out, c.widths, c.rank, backward)
        whole = torch.full((nbytes + (1 << 20),), 0xA7, dtype=torch.uint8, device="cuda")
        r.workspace = whole[:nbytes]
        r.forward()
        if backward:
            r.backward()
        got = r.outputs()
        test_mx.check(c, got, ("y", "s", "dx", "da", "db", "dbias", "u") if backward else ("y", "s"))
        assert (whole[nbytes:] == 0xA7).all()
