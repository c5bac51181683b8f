"""Infinite weights, activations and logits give what the formulas give: an
infinity of the right sign where one term of a sum is infinite, NaN only where
the formula has it (infinities of both signs, 0 times infinity)."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(__file__))
import test_linear as linear  # noqa: E402
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


# (tokens, hidden, widths): 64 x 64 tiles, and 256 x 256 ones of y and dx
SIZES = [(20, 136, [136, 40]), (300, 136, [136, 40]), (2050, 136, [5400, 72]), (2050, 5400, [72, 40])]


@pytest.mark.gpu
@pytest.mark.parametrize("n,hidden,widths", SIZES)
@pytest.mark.parametrize("rank", [8, 16, 24, 32, 72, 128])
def test_infinite_adapter_weights(n, hidden, widths, rank):
    """One infinite entry of B is an infinite column of y for the adapter's
    tokens, with the sign of s; one of A, an infinite column of dx with the sign of u."""
    c = linear.Case(n=n, hidden=hidden, widths=widths, rank=rank, loras=2)
    r = linear.Run(c)
    r.forward()
    r.backward()
    clean = r.outputs()
    mine = c.ids == 1
    col, row = widths[0] - 3, hidden - 5
    r.b[0][1, col, rank - 1] = INF
    r.forward()
    y = r.outputs()["y"]
    want = clean["y"].clone()
    want[mine, col] = INF * clean["s"][0][mine, rank - 1].sign()
    assert torch.equal(y[mine, col], want[mine, col])
    same = torch.ones(c.out, dtype=torch.bool)
    same[col] = False
    assert torch.isfinite(y[:, same]).all() and torch.isfinite(y[~mine]).all()
    r.b[0][1, col, rank - 1] = 1.0
    r.backward()                                  # u of a finite B again
    u = r.outputs()["u"][0]
    r.a[0][1, rank - 1, row] = -INF
    r.backward()
    dx = r.outputs()["dx"]
    assert torch.equal(dx[mine, row], -INF * u[mine, rank - 1].sign())
    same = torch.ones(hidden, dtype=torch.bool)
    same[row] = False
    assert torch.isfinite(dx[:, same]).all() and torch.isfinite(dx[~mine]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("n,loras", [(20, 2), (300, 2), (1100, 3)])
@pytest.mark.parametrize("rank", [8, 24, 64])
def test_infinite_activations(n, loras, rank):
    """One infinite entry of x or dy is an infinite column of dA or dB of its
    token's adapter, with the signs of the token's u or s."""
    c = linear.Case(n=n, hidden=136, widths=[136, 40], rank=rank, loras=loras)
    r = linear.Run(c)
    r.forward()
    r.backward()
    clean = r.outputs()
    t = int(torch.nonzero(c.ids == 1)[2])
    h, col = 100, 30
    r.x[t, h] = INF                               # s is the forward pass's of before
    r.backward()
    da = r.outputs()["da"]
    for i in range(2):
        assert torch.equal(da[i][1, :, h], INF * clean["u"][i][t].sign())
        da[i][1, :, h] = 0.0
        assert torch.isfinite(da[i]).all()
    r.x[t, h] = 1.0
    r.dy[t, col] = -INF
    r.backward()
    got = r.outputs()
    assert torch.equal(got["db"][0][1, col], -INF * clean["s"][0][t].sign())
    assert got["dbias"][0][1, col] == -INF
    got["db"][0][1, col] = 0.0
    assert all(torch.isfinite(v).all() for v in got["db"])
