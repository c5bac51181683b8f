"""A loss whose tiles do not fit one launch: tokens at both ends and on both sides
of the edge, against the formula in 64 bits; tolerances as in test_loss."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(__file__))
import test_loss as loss  # noqa: E402

U8, U22, U23 = 2.0 ** -8, 2.0 ** -22, 2.0 ** -23
SLACK = 1 + 2.0 ** -6


def _normal(*shape, sigma=1.0):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, sigma)


STEP = 1 << 20   # vocabulary entries of a reference product (each far below 2^31 elements)


def _logits(x, w):
    """x w^T in 64 bits, and the largest sum of magnitudes of each token."""
    parts, size = [], torch.zeros(x.shape[0], dtype=torch.float64, device="cuda")
    for lo in range(0, w.shape[0], STEP):
        wd = w[lo:lo + STEP].double()
        parts.append(x @ wd.t())
        size = torch.maximum(size, (x.abs() @ wd.abs().t()).max(1).values)
    return torch.cat(parts, 1), size


def _lse_bound(hidden, z, size):
    """test_loss's bound of lse."""
    top, lse = z.max(1).values, torch.logsumexp(z, 1)
    own = torch.stack([(torch.exp(a - b) * U22 * ((a - t).abs() + 4)).sum() for a, b, t in zip(z, lse, top)])
    return (U23 * (hidden + 8) * size + own + U23 * (256 + z.shape[1] / 2048) + U22 * (lse.abs() + top.abs() + 1)) * SLACK


@pytest.mark.gpu
def test_loss_in_more_than_one_launch():
    """65536 by 129 tiles: more threads than a launch may have."""
    sgl = loss.lib()
    torch.manual_seed(4)
    n, hidden, vocab = 33000, 8, 1 << 24
    x, w = _normal(n, hidden), _normal(vocab, hidden, sigma=0.5)
    targets = torch.randint(0, vocab, (n,), dtype=torch.int32, device="cuda")
    targets[7], targets[n - 1] = -1, vocab - 1
    got, lse = (torch.full((n,), float("nan"), device="cuda") for _ in range(2))
    ws = torch.empty(sgl.lora_cross_entropy_workspace_bytes(n, hidden, vocab), dtype=torch.uint8, device="cuda")
    sgl.lora_cross_entropy(x, w, targets, got, lse, ws)
    torch.cuda.synchronize()
    del ws
    assert torch.isfinite(got).all() and torch.isfinite(lse).all() and got[7] == 0
    at = torch.tensor([0, 255, 256, 32511, 32512, 32513, n - 233, n - 1], device="cuda")   # 127 tiles of 256 tokens a launch
    z, size = _logits(x[at].double(), w)
    want, bound = torch.logsumexp(z, 1), _lse_bound(hidden, z, size)
    assert ((lse[at].double() - want).abs() <= bound).all()
    assert ((got[at].double() - (want - z.gather(1, targets[at].long()[:, None])[:, 0])).abs() <= 2 * bound).all()
