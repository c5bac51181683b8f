"""Tensors of more than 2^31 elements, and a loss whose tiles do not fit one launch:
rows at both ends and on both sides of the edges, against the formulas in 64
bits; tolerances as in test_linear and test_loss."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(__file__))
import test_linear as linear  # noqa: E402
import test_loss as loss  # noqa: E402

U8, U22, U23 = 2.0 ** -8, 2.0 ** -22, 2.0 ** -23
SLACK = 1 + 2.0 ** -6


def _normal(*shape, sigma=1.0):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, sigma)


class Rows:
    """Some of a large batch's tokens as a case of their own (y and dx are row by row)."""

    def __init__(self, r, at):
        host = lambda t: t.cpu()
        self.n, self.hidden, self.widths, self.rank, self.loras = len(at), r.x.shape[1], r.widths, r.rank, r.loras
        self.offset, self.out, self.scale = 0, r.w.shape[0], r.scale
        self.ids, self.x, self.dy = host(r.ids[at]), host(r.x[at]), host(r.dy[at])
        self.w, self.a, self.b = host(r.w), [host(t) for t in r.a], [host(t) for t in r.b]
        self.w_bias = self.bias = None


class Large:
    def __init__(self, n, hidden, widths, rank, loras):
        sgl = linear.lib()
        torch.manual_seed(3)
        self.widths, self.rank, self.loras, self.scale = widths, rank, loras, 0.5
        out = sum(widths)
        self.x, self.dy, self.w = _normal(n, hidden), _normal(n, out, sigma=0.1), _normal(out, hidden, sigma=0.05)
        self.a = [_normal(loras, rank, hidden, sigma=0.05) for _ in widths]
        self.b = [_normal(loras, w, rank, sigma=0.05) for w in widths]
        self.ids = torch.randint(-1, loras, (n,), dtype=torch.int32, device="cuda")
        self.meta = sgl.LoraMeta(loras, n)
        sgl.lora_prepare_meta(self.ids, self.meta)
        buf, dbuf = (torch.empty(len(widths), n, rank, device="cuda") for _ in range(2))
        self.y, self.dx = torch.empty_like(self.dy), torch.empty_like(self.x)
        self.da, self.db = [torch.empty_like(t) for t in self.a], [torch.empty_like(t) for t in self.b]
        ws = torch.empty(sgl.lora_linear_workspace_bytes(n, loras, hidden, widths, rank, True), dtype=torch.uint8, device="cuda")
        sgl.lora_linear(self.x, self.w, None, self.a, self.b, None, buf, self.y, self.meta, self.scale, ws)
        sgl.lora_linear_backward(self.dy, self.x, self.w, self.a, self.b, buf, dbuf, self.dx, self.da, self.db, None,
                                 self.meta, self.scale, ws)
        self.buf, self.dbuf = buf, dbuf


@pytest.mark.gpu
@pytest.mark.parametrize("hidden,widths", [(64, [32000, 768]), (32768, [40, 24])])
def test_linear_past_31_bits(hidden, widths):
    n = 70000
    r = Large(n, hidden, widths, 8, 3)
    assert max(r.y.numel(), r.x.numel()) > 2 ** 31
    edge = 2 ** 31 // max(hidden, sum(widths))      # the row with element 2^31
    at = torch.tensor([0, 1, 255, 256, edge - 1, edge, edge + 1, n - 257, n - 2, n - 1], device="cuda")
    c = Rows(r, at)
    val, mag = linear.reference(c)
    tol = linear.tolerances(c, val, mag)
    for k, got in (("y", r.y[at]), ("dx", r.dx[at])):
        assert ((got.cpu().double() - val[k]).abs() <= tol[k]).all(), k
    # gradients of one adapter from its own s and u: the last columns
    m, mine = 1, r.ids == 1
    x, dy = r.x[:, -40:][mine].double(), r.dy[:, -16:][mine].double()
    u, s = r.dbuf[-1][mine].double(), r.buf[-1][mine].double()
    count = int(mine.sum())
    for got, p, q in ((r.da[-1][m][:, -40:], u, x), (r.db[-1][m][-16:], dy, s)):
        want, size = p.t() @ q, p.abs().t() @ q.abs()
        assert ((got.double() - want).abs() <= U8 * want.abs() + (2.0 ** -16 + U23 * (2 * count + 8)) * size * SLACK).all()


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


@pytest.mark.gpu
def test_loss_past_31_bits():
    """A vocabulary matrix and its gradient of 2.3e9 elements, in several pieces."""
    sgl = loss.lib()
    torch.manual_seed(5)
    n, hidden, vocab = 40, 136, 1 << 24
    x, w = _normal(n, hidden), _normal(vocab, hidden, sigma=0.05)
    targets = torch.randint(0, vocab, (n,), dtype=torch.int32, device="cuda")
    edge = 2 ** 31 // hidden
    targets[0], targets[1], targets[2], targets[3] = 0, edge, vocab - 1, -1
    dl = torch.randn(n, device="cuda")
    got, lse = (torch.empty(n, device="cuda") for _ in range(2))
    dx, dw = torch.empty_like(x), torch.full_like(w, float("nan"))
    ws = torch.empty(sgl.lora_cross_entropy_workspace_bytes(n, hidden, vocab, True), dtype=torch.uint8, device="cuda")
    sgl.lora_cross_entropy(x, w, targets, got, lse, ws)
    sgl.lora_cross_entropy_backward(x, w, targets, lse, dl, dx, dw, ws)
    torch.cuda.synchronize()
    del ws
    assert all(torch.isfinite(dw[lo:lo + STEP]).all() for lo in range(0, vocab, STEP))
    xd = x.double()
    z, size = _logits(xd, w)
    want, bound = torch.logsumexp(z, 1), _lse_bound(hidden, z, size)
    assert ((lse.double() - want).abs() <= bound).all()
    on = targets >= 0
    scale = torch.where(on, dl, torch.zeros_like(dl)).double()[:, None]
    hot = torch.where(on, targets, torch.zeros_like(targets)).long()[:, None]
    value, limit = (torch.zeros(n, hidden, dtype=torch.float64, device="cuda") for _ in range(2))
    at = torch.cat([torch.tensor([0, 1, edge - 1, edge, edge + 1, vocab - 2, vocab - 1], device="cuda"), targets[4:20].long()])
    for lo in range(0, vocab, STEP):
        wd, arg = w[lo:lo + STEP].double(), z[:, lo:lo + STEP] - want[:, None]
        p = torch.exp(arg)
        here = ((hot >= lo) & (hot < lo + STEP)).double()
        g = scale * p.scatter_add(1, (hot - lo).clamp(0, STEP - 1), -here)
        eg = U8 * g.abs() + scale.abs() * (p * ((U23 * (hidden + 8) * size + bound)[:, None] + U22 * (arg.abs() + 4)) + U23)
        value += g @ wd
        limit += eg @ wd.abs() + U23 * (vocab + 8) * (g.abs() @ wd.abs())
        rows = at[(at >= lo) & (at < lo + STEP)]
        if len(rows):
            gr, er = g[:, rows - lo].t().contiguous(), eg[:, rows - lo].t().contiguous()
            wants = gr @ xd
            bounds = U8 * wants.abs() + er @ xd.abs() + U23 * (n + 8) * (gr.abs() @ xd.abs())
            assert ((dw[rows].double() - wants).abs() <= bounds * SLACK).all(), rows.tolist()
    assert ((dx.double() - value).abs() <= (U8 * value.abs() + limit) * SLACK).all()
