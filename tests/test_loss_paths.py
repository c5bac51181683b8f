"""lora_cross_entropy and its backward pass at the sizes where another tile is
chosen, against the formulas in 64 bits; inputs, references and tolerances as in
test_loss."""
import os
import sys

import pytest

sys.path.insert(0, os.path.dirname(__file__))
from test_loss import Case, Run, check  # noqa: E402

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
