"""The loss of tokens whose target is nearly certain, or far from it, at large
logits: its digits are those of (max - z[target]) + log sum exp(z - max), not of
a rounded lse less z[target].

All but eight entries of the vocabulary have logits so low that their
exponentials are zeros, and every product is exact in float32, so that what is
off is (2^-24: half a step of float32):
  exp  : 2^-22 (|argument| + 4) of the value, once in a tile and once where tiles are joined
  sum  : at most 8 terms that are not zero, an addition of each within a tile and
         one where tiles are joined: 16 * 2^-24 of the sum
  log  : 2^-22 of the value
  loss : its addition and its difference, 2^-24 of each
"""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(__file__))
from test_loss import lib  # noqa: E402

U22, U24 = 2.0 ** -22, 2.0 ** -24


def inputs(n, vocab, seed=0):
    """Logits x[t][0] * w[v][0]: 64, 60, 56, ... for eight entries, below -100 for the others."""
    g = torch.Generator().manual_seed(seed + 7 * n + vocab)
    few = min(8, vocab)
    x, w = torch.zeros(n, 8), torch.zeros(vocab, 8)
    x[:, 0] = torch.tensor([0.5, 0.75, 0.875, 1.0])[torch.randint(0, 4, (n,), generator=g)]
    w[:, 0] = -256.0
    at = torch.randperm(vocab, generator=g)[:few]
    w[at, 0] = 64.0 - 4.0 * torch.arange(few) - torch.randint(0, 4, (few,), generator=g)
    # targets: the largest entry, and each of the others
    targets = at[torch.where(torch.arange(n) % 2 == 0, torch.zeros(n, dtype=torch.long), torch.arange(n) % few)]
    return x.to(torch.bfloat16), w.to(torch.bfloat16), targets.to(torch.int32)


@pytest.mark.gpu
@pytest.mark.parametrize("n,vocab", [(1, 8), (20, 2003), (64, 8), (200, 5003), (300, 24600)])
def test_loss_keeps_its_digits(n, vocab):
    sgl = lib()
    x, w, targets = inputs(n, vocab)
    loss, lse = (torch.full((n,), float("nan"), device="cuda") for _ in range(2))
    workspace = torch.zeros(sgl.lora_cross_entropy_workspace_bytes(n, 8, vocab), dtype=torch.uint8, device="cuda")
    sgl.lora_cross_entropy(x.cuda(), w.cuda(), targets.cuda(), loss, lse, workspace)
    z = x.double() @ w.double().t()
    top = z.max(1, keepdim=True).values
    terms = (z - top).exp()
    total = terms.sum(1)
    gap = top[:, 0] - z.gather(1, targets.long()[:, None])[:, 0]
    # (log1p of the terms but the largest: 64 bits would lose digits of its own)
    rest = terms.scatter(1, z.argmax(1, keepdim=True), 0.0).sum(1)
    want = gap + torch.log1p(rest)
    off = (terms * 2 * U22 * ((z - top).abs() + 4) * (z < top)).sum(1) / total + 16 * U24 + U22 * total.log()
    tol = (off + U24 * (gap + want)) * (1 + 2.0 ** -6)
    worst = ((loss.cpu().double() - want).abs() / tol).max().item()
    assert worst <= 1, "%.3g times the tolerance" % worst
    assert ((lse.cpu().double() - torch.logsumexp(z, 1)).abs() <= off + U24 * 2 * 64).all()
