"""lora_cross_entropy and lora_cross_entropy_backward against the formulas in
64 bits on the CPU.

Tolerances, derived from the arithmetic.  With M(x w) = sum_k |x||w|:
  z    : e_z = 2^-23 (H + 8) M(x w)      (float32 sums; the matrix unit may truncate)
  exp  : 2^-22 (|argument| + 4) of the value (rounded argument, the hardware's 2^x)
  lse  : e_l = max_v e_z + sum_v p_v 2^-22 (|z - max| + 4) + 2^-23 (256 + V / 2048) + 2^-22 (|lse| + |max| + 1)
         (sums of exponentials: at most 256 additions within a tile and its joins, then the tiles')
  loss : e_l + e_z[target] + 2^-23 (|loss| + |lse|)
  g    : 2^-8 |g| (bfloat16) + |dloss| (p (e_z + e_l + 2^-22 (|z - lse| + 4)) + 2^-23)
  dx   : 2^-8 |dx| + sum_v e_g |w| + 2^-23 (V + 8) sum_v |g||w|;  dw with the tokens and x
times 1 + 2^-6 for the products of these factors.
"""
import ctypes
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(__file__))

U8, U22, U23 = 2.0 ** -8, 2.0 ** -22, 2.0 ** -23
SLACK = 1 + 2.0 ** -6


def lib():
    from segmented_gather_lora_amd import _build
    _build.ensure_built()
    import segmented_gather_lora_amd as sgl
    return sgl


class Case:
    def __init__(self, n, hidden, vocab, ignored=0.2, seed=0, sure=8.0, stride=0, sigma=0.05):
        g = torch.Generator().manual_seed(1013 * seed + 31 * n + vocab)
        self.n, self.hidden, self.vocab, self.stride = n, hidden, vocab, stride
        self.w = (torch.randn(vocab, hidden, generator=g) * sigma).to(torch.bfloat16)
        targets = torch.randint(0, vocab, (n,), generator=g)
        rows = self.w[targets].float()
        lift = sure * torch.rand(n, 1, generator=g)
        x = torch.randn(n, hidden, generator=g)
        self.x = (x + lift * rows / (rows * rows).sum(1, keepdim=True).clamp(min=1e-3)).to(torch.bfloat16)
        targets[torch.rand(n, generator=g) < ignored] = -1
        self.targets = targets.to(torch.int32)
        self.dloss = torch.randn(n, generator=g)


def reference(c):
    x, w, dl = c.x.double(), c.w.double(), c.dloss.double()
    on = (c.targets >= 0) & (c.targets < c.vocab)
    at = torch.where(on, c.targets.long(), torch.zeros_like(c.targets.long()))[:, None]
    z, ez = x @ w.t(), U23 * (c.hidden + 8) * (x.abs() @ w.abs().t())
    top = z.max(1, keepdim=True).values
    lse = torch.logsumexp(z, 1)
    p = torch.exp(z - lse[:, None])
    loss = torch.where(on, lse - z.gather(1, at)[:, 0], torch.zeros_like(lse))
    el = (ez.max(1).values + (p * U22 * ((z - top).abs() + 4)).sum(1) + U23 * (256 + c.vocab / 2048)
          + U22 * (lse.abs() + top[:, 0].abs() + 1))
    hot = torch.zeros_like(p).scatter_(1, at, 1.0)
    g = torch.where(on[:, None], (p - hot) * dl[:, None], torch.zeros_like(p))
    eg = U8 * g.abs() + on[:, None] * dl.abs()[:, None] * (p * (ez + el[:, None] + U22 * ((z - lse[:, None]).abs() + 4)) + U23)
    val = {"loss": loss, "lse": lse, "dx": g @ w, "dw": g.t() @ x}
    xf = torch.where(on[:, None], x, torch.zeros_like(x))
    tol = {"lse": el, "loss": el + ez.gather(1, at)[:, 0] + U23 * (loss.abs() + lse.abs()),
           "dx": U8 * val["dx"].abs() + eg @ w.abs() + U23 * (c.vocab + 8) * (g.abs() @ w.abs()),
           "dw": U8 * val["dw"].abs() + eg.t() @ xf.abs() + U23 * (c.n + 8) * (g.abs().t() @ xf.abs())}
    return val, {k: v * SLACK + 1e-37 for k, v in tol.items()}, g


class Run:
    def __init__(self, c, poison=float("nan")):
        sgl = lib()
        self.c = c

        def strided(t):
            if not c.stride:
                return t.cuda()
            wide = torch.full((t.shape[0], t.shape[1] + c.stride), float("nan"), dtype=t.dtype, device="cuda")
            wide[:, :t.shape[1]] = t.cuda()
            return wide[:, :t.shape[1]]
        self.x, self.w = strided(c.x), strided(c.w)
        self.targets, self.dloss = c.targets.cuda(), c.dloss.cuda()
        f = lambda *s: torch.full(s, poison, dtype=torch.float32, device="cuda")
        self.loss, self.lse = f(c.n), f(c.n)
        self.dx = strided(torch.full((c.n, c.hidden), poison, dtype=torch.bfloat16))
        self.dw = strided(torch.full((c.vocab, c.hidden), poison, dtype=torch.bfloat16))
        # the workspace's contents do not matter
        self.workspace = torch.full((sgl.lora_cross_entropy_workspace_bytes(c.n, c.hidden, c.vocab, True),), 0xff,
                                    dtype=torch.uint8, device="cuda")

    def forward(self, **kw):
        lib().lora_cross_entropy(self.x, self.w, self.targets, self.loss, self.lse, self.workspace, **kw)

    def status(self):
        return int(self.workspace[:4].view(torch.int32).item())

    def backward(self, dx=True, dw=True, **kw):
        lib().lora_cross_entropy_backward(self.x, self.w, self.targets, self.lse, self.dloss, self.dx if dx else None,
                                          self.dw if dw else None, self.workspace, **kw)

    def outputs(self):
        torch.cuda.synchronize()
        return {k: getattr(self, k).cpu().double() for k in ("loss", "lse", "dx", "dw")}


def check(c, got, keys=("loss", "lse", "dx", "dw")):
    val, tol, _ = reference(c)
    for k in keys:
        assert torch.isfinite(got[k]).all(), "%s has values that are not finite" % k
        worst = ((got[k] - val[k]).abs() / tol[k]).max().item() if got[k].numel() else 0.0
        assert worst <= 1, "%s: %.3g times the tolerance" % (k, worst)
    off = (c.targets < 0) | (c.targets >= c.vocab)
    assert (got["loss"][off] == 0).all()
    if "dx" in keys:
        assert (got["dx"][off] == 0).all()


CASES = {
    "one token": dict(n=1, hidden=72, vocab=1000, ignored=0.0),
    "one ignored token": dict(n=1, hidden=64, vocab=130, ignored=1.0),
    "vocabulary of one": dict(n=5, hidden=8, vocab=1, ignored=0.0),
    "vocabulary of seven": dict(n=40, hidden=16, vocab=7),
    "16": dict(n=16, hidden=1032, vocab=4099, ignored=0.0),
    "32": dict(n=32, hidden=264, vocab=513),
    "33": dict(n=33, hidden=136, vocab=385, stride=8),
    "129": dict(n=129, hidden=72, vocab=5003),
    "all ignored": dict(n=70, hidden=72, vocab=300, ignored=1.0),
    "one counts": dict(n=300, hidden=64, vocab=257, ignored=0.997),
    "sure": dict(n=64, hidden=264, vocab=2000, sure=60.0),
    "large logits": dict(n=50, hidden=520, vocab=900, sigma=2.0, sure=0.0),
    "few classes, many tokens": dict(n=1500, hidden=200, vocab=100),
    "several pieces": dict(n=17, hidden=16, vocab=9001),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(CASES))
def test_against_formulas(name):
    c = Case(**CASES[name])
    r = Run(c)
    r.forward()
    assert r.status() == 0
    r.backward()
    first = r.outputs()
    check(c, first)
    r.forward()
    r.backward()
    again = r.outputs()
    assert all(torch.equal(first[k], again[k]) for k in first)


@pytest.mark.gpu
@pytest.mark.parametrize("n,hidden,vocab", [(2049, 72, 6000), (600, 1032, 16600), (4100, 3080, 300)])
def test_large_tiles(n, hidden, vocab):
    c = Case(n=n, hidden=hidden, vocab=vocab, ignored=0.3)
    r = Run(c)
    r.forward()
    r.backward()
    check(c, r.outputs())


@pytest.mark.gpu
def test_pieces_of_the_vocabulary():
    """40000 tokens: g's buffer holds 4096 vocabulary rows, so the vocabulary
    takes three pieces (the last one ragged)."""
    c = Case(n=40000, hidden=8, vocab=8500, ignored=0.3)
    r = Run(c)
    assert r.workspace.numel() < 2 * 40000 * 4608 + 8 * 40000 * (8500 // 128 + 64)
    r.forward()
    r.backward()
    check(c, r.outputs())


@pytest.mark.gpu
def test_empty_batch():
    c = Case(n=0, hidden=16, vocab=300)
    r = Run(c)
    r.forward()
    r.backward()
    assert (r.outputs()["dw"] == 0).all()


@pytest.mark.gpu
def test_optional_gradients():
    c = Case(n=40, hidden=72, vocab=600)
    r = Run(c)
    r.forward()
    r.backward(dw=False)
    got = r.outputs()
    check(c, got, ("loss", "lse", "dx"))
    assert torch.isnan(got["dw"]).all()
    r = Run(c)
    r.forward()
    r.backward(dx=False)
    got = r.outputs()
    check(c, got, ("loss", "lse", "dw"))
    assert torch.isnan(got["dx"]).all()


@pytest.mark.gpu
def test_targets_out_of_range():
    c = Case(n=20, hidden=64, vocab=200, ignored=0.0)
    c.targets[3], c.targets[7], c.targets[11] = 200, -7, 2 ** 31 - 1
    r = Run(c)
    r.forward()
    assert r.status() == lib().LORA_ERR_ID_RANGE
    r.backward()
    check(c, r.outputs())


@pytest.mark.gpu
def test_ignored_tokens_may_hold_anything():
    """x, lse and dloss of ignored tokens that are not finite reach nothing else."""
    c = Case(n=150, hidden=72, vocab=700, ignored=0.3)
    off = c.targets < 0
    r = Run(c)
    r.forward()
    r.backward()
    clean = r.outputs()
    r.x[off.cuda()] = float("nan")
    r.dloss[off.cuda()] = float("inf")
    r.forward()
    r.backward()
    got = r.outputs()
    assert torch.equal(got["loss"], clean["loss"]) and torch.equal(got["lse"][~off], clean["lse"][~off])
    assert torch.equal(got["dx"], clean["dx"]) and torch.equal(got["dw"], clean["dw"])


@pytest.mark.gpu
def test_masked_vocabulary():
    """Rows of the type's lowest value and of minus infinity leave the others' softmax."""
    c = Case(n=30, hidden=16, vocab=400, ignored=0.0)
    c.x[:, 0] = 1.0
    c.x = c.x.abs()
    c.w[:, 0] = 0.0
    keep = torch.ones(400, dtype=torch.bool)
    keep[5:60] = False
    c.targets = torch.full((30,), 399, dtype=torch.int32)
    c.w[~keep] = 0.0
    c.w[5:40, 0] = torch.finfo(torch.bfloat16).min
    c.w[40:60, 0] = float("-inf")
    r = Run(c)
    r.forward()
    got = r.outputs()
    z = c.x.double() @ c.w[keep].double().t()
    want = torch.logsumexp(z, 1)
    assert ((got["lse"] - want).abs() <= 1e-4 * (1 + want.abs())).all()
    assert ((got["loss"] - (want - z[:, -1])).abs() <= 1e-4 * (1 + want.abs())).all()


@pytest.mark.gpu
def test_gradients_against_differences():
    c = Case(n=40, hidden=64, vocab=300, sure=3.0)
    r = Run(c)
    r.forward()
    r.backward()
    got = r.outputs()
    _, tol, _ = reference(c)
    on = c.targets >= 0
    at = c.targets.clamp(min=0).long()[:, None]
    gen = torch.Generator().manual_seed(3)

    def total(x, w):
        z = x @ w.t()
        return ((torch.logsumexp(z, 1) - z.gather(1, at)[:, 0]) * c.dloss.double() * on).sum().item()
    x, w, h = c.x.double(), c.w.double(), 1e-4
    for key, base in (("dx", x), ("dw", w)):
        step = torch.randn(base.shape, generator=gen, dtype=torch.float64)
        moved = [(x + s * h * step, w) if key == "dx" else (x, w + s * h * step) for s in (1, -1)]
        diff = (total(*moved[0]) - total(*moved[1])) / (2 * h)
        # the differences' own error: third derivatives, h^2 times the cube of the steps' logits
        size = (step.abs() @ w.abs().t() if key == "dx" else x.abs() @ step.abs().t()).max().item()
        own = h * h * size ** 3 * c.dloss.abs().sum().item()
        assert abs((got[key] * step).sum().item() - diff) <= (tol[key] * step.abs()).sum().item() + own


@pytest.mark.gpu
def test_other_stream_and_graph_replays():
    c = Case(n=90, hidden=264, vocab=3001)
    r = Run(c)
    r.forward()
    r.backward()
    eager = r.outputs()
    check(c, eager)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        r.forward()
        r.backward()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(v, eager[k]) for k, v in r.outputs().items())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r.forward()
        r.backward()
    for _ in range(4):
        for t in (r.loss, r.lse, r.dx, r.dw):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(v, eager[k]) for k, v in r.outputs().items())
        r.x.mul_(1.0)


# ------------------------------------------------------------------ refusals (no GPU)

def test_refusals():
    sgl = lib()
    L = sgl.lib
    assert sgl.lora_cross_entropy_workspace_bytes(16, 64, 1000) <= sgl.lora_cross_entropy_workspace_bytes(16, 64, 1000, True)
    for bad in ((-1, 64, 10), (1, 60, 10), (1, 0, 10), (1, 64, 0), (1, 64, 16777217)):
        assert L.lora_cross_entropy_workspace_bytes(*bad, 1) == 0
    with pytest.raises(sgl.LoraError):
        sgl.lora_cross_entropy_workspace_bytes(1, 60, 10)
    need = sgl.lora_cross_entropy_workspace_bytes(16, 64, 1000, True)
    ok = dict(x=0x10000, ldx=64, n=16, h=64, w=0x20000, ldw=64, v=1000, t=0x30000, loss=0x40000, lse=0x50000, dl=0x60000,
              dx=0x70000, lddx=64, dw=0x80000, lddw=64, ws=0x90000, nb=need)

    def fwd(**kw):
        a = dict(ok, **kw)
        return L.lora_cross_entropy(a["x"], a["ldx"], a["n"], a["h"], a["w"], a["ldw"], a["v"], a["t"], a["loss"],
                                    a["lse"], a["ws"], a["nb"], None)

    def bwd(**kw):
        a = dict(ok, **kw)
        return L.lora_cross_entropy_backward(a["x"], a["ldx"], a["n"], a["h"], a["w"], a["ldw"], a["v"], a["t"],
                                             a["lse"], a["dl"], a["dx"], a["lddx"], a["dw"], a["lddw"], a["ws"],
                                             a["nb"], None)
    for call in (fwd, bwd):
        assert call(n=-1) == sgl.LORA_ERR_NUM_TOKENS
        for kw in (dict(h=60), dict(ldx=56), dict(ldx=68), dict(ldw=56), dict(v=0)):
            assert call(**kw) == sgl.LORA_ERR_SHAPE, kw
        for kw in (dict(x=None), dict(w=None), dict(t=None), dict(lse=None), dict(ws=None)):
            assert call(**kw) == sgl.LORA_ERR_NULL, kw
        for kw in (dict(x=0x10008), dict(w=0x20002)):
            assert call(**kw) == sgl.LORA_ERR_ALIGN, kw
        assert call(ws=0x90010) == sgl.LORA_ERR_BUFFER and call(nb=100) == sgl.LORA_ERR_BUFFER
    assert fwd(loss=None) == sgl.LORA_ERR_NULL and bwd(dl=None) == sgl.LORA_ERR_NULL
    assert bwd(lddx=56) == sgl.LORA_ERR_SHAPE and bwd(lddw=68) == sgl.LORA_ERR_SHAPE
    assert bwd(dx=0x70008) == sgl.LORA_ERR_ALIGN and bwd(dw=0x80008) == sgl.LORA_ERR_ALIGN
    assert fwd(n=0) == sgl.LORA_OK and bwd(dx=None, dw=None) == sgl.LORA_OK


def test_binding_refuses_what_the_library_cannot_see():
    sgl = lib()
    x, w = torch.zeros(4, 16, dtype=torch.bfloat16), torch.zeros(9, 16, dtype=torch.bfloat16)
    t, f, ws = torch.zeros(4, dtype=torch.int32), torch.zeros(4), torch.zeros(64, dtype=torch.uint8)
    with pytest.raises(TypeError):
        sgl.lora_cross_entropy(x, w, t, f, f, ws)
    with pytest.raises(TypeError):
        sgl.lora_cross_entropy_backward(x, w, t, f, f, None, None, ws)
