"""Infinite logits give what the formulas give: an infinity of the right sign
where one term of a sum is infinite, NaN only where the formula has it."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(__file__))
import test_loss as loss  # noqa: E402

INF = float("inf")

LOGITS = [(7, 300), (20, 5003), (64, 1000), (300, 24600)]


@pytest.mark.gpu
@pytest.mark.parametrize("n,vocab", LOGITS)
def test_infinite_logits(n, vocab):
    """An entry of +inf: lse and every other target's loss are +inf; tokens for
    which the same entry is -inf lose that entry alone."""
    c = loss.Case(n=n, hidden=72, vocab=vocab, ignored=0.0)
    bad = vocab // 2
    c.w[bad, 3] = INF
    c.x[:, 3] = torch.where(torch.arange(n) % 3 == 0, torch.tensor(-1.0), torch.tensor(0.5)).to(torch.bfloat16)
    c.targets[c.targets == bad] = bad + 1
    if n > 4:
        c.targets[4] = bad                       # +inf - +inf
    r = loss.Run(c)
    r.forward()
    got = r.outputs()
    up = c.x[:, 3] > 0
    on = torch.ones(n, dtype=torch.bool)
    on[4] = False
    assert (got["lse"][up] == INF).all() and (got["loss"][up & on] == INF).all()
    assert torch.isnan(got["loss"][4])
    keep = torch.arange(vocab) != bad
    z = c.x.double() @ c.w[keep].double().t()
    want = torch.logsumexp(z, 1)
    assert ((got["lse"] - want).abs() <= 1e-4 * (1 + want.abs()))[~up].all()
