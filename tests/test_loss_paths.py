"""lora_cross_entropy and its backward pass at the sizes where another tile is
chosen, against the formulas in 64 bits; inputs, references and tolerances as in
test_loss."""
import os
import sys

import pytest

sys.path.insert(0, os.path.dirname(__file__))
from test_loss import Case, Run, check, lib, reference  # noqa: E402

CASES = {
    "128 x 128": dict(n=200, hidden=2056, vocab=25001),
    "64 x 64": dict(n=130, hidden=72, vocab=1003),
    "64 x 64, few entries": dict(n=70, hidden=264, vocab=3),
    "128 x 32": dict(n=31, hidden=136, vocab=9001),
    "128 x 32, one step": dict(n=5, hidden=64, vocab=260),
    "256 x 256, one step": dict(n=513, hidden=56, vocab=20003),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(CASES))
def test_tiles(name):
    c = Case(**CASES[name])
    r = Run(c)
    r.forward()
    r.backward()
    check(c, r.outputs())


@pytest.mark.gpu
@pytest.mark.parametrize("n,vocab,head", [(1, 1000, 0), (70, 40, 3), (700, 5003, 1), (2100, 300, 0)])
def test_gradients_of_targets_are_not_rounded_twice(n, vocab, head):
    """The rounding of g to bfloat16 alone is off by up to 2^-8 of the target's
    entry, which is most of g: rms errors stay at what the rounding of the
    result itself can cost (2^-8, half a step) less the average (1 / sqrt(3))."""
    c = Case(n=n, hidden=264, vocab=vocab, ignored=0.0, sure=6.0)
    if head:      # many tokens of few targets: more than one K step of them in a tile
        c.targets = c.targets % head
    r = Run(c)
    r.forward()
    r.backward()
    got = r.outputs()
    check(c, got)
    val, _, _ = reference(c)
    for k in ("dx", "dw"):
        err = (got[k] - val[k]).norm() / val[k].norm()
        assert err <= 2.0 ** -8 / 3 ** 0.5, (k, err)


def test_widths_past_the_limit_are_refused():
    sgl = lib()
    assert sgl.lora_cross_entropy_workspace_bytes(1, 1 << 24, 8) > 0
    with pytest.raises(sgl.LoraError):
        sgl.lora_cross_entropy_workspace_bytes(1, (1 << 24) + 8, 8)
