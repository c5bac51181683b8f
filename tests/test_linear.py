"""lora_linear and lora_linear_backward: the shared projection with adapters and
its gradients, against the formulas in 64 bits on the CPU.

Tolerances, derived from the arithmetic.  A rounding to bfloat16 is off by at
most 2^-8 of the value; a float32 sum of k products by at most k * 2^-23 of the
sum of their magnitudes (2^-23: the matrix unit's additions may truncate); the
two bfloat16 parts of s and u together by at most 2^-16 of the value.  With
M(.) the same expression over magnitudes and S, U those of s and u:
  y   : 2^-8 |y| + 2^-23 (H + 8) M(x w)  + (2^-16 + 2^-23 (H + 2 r + 8)) M(S b)
  dx  : 2^-8 |dx| + 2^-23 (O + 8) M(dy w) + (2^-16 + 2^-23 (w + 2 r + 8)) M(U a)
  da  : 2^-8 |da| + (2^-16 + 2^-23 (w + 2 n + 8)) M(U x);  db with H, S, dy
  dbias: 2^-8 |dbias| + 2^-23 (n + 8) M(dy)
times 1 + 2^-6 for the products of these factors.
"""
import ctypes
import math
import os
import sys

import numpy as np
import pytest
import torch

sys.path.insert(0, os.path.dirname(__file__))

U8, U16, U23 = 2.0 ** -8, 2.0 ** -16, 2.0 ** -23
SLACK = 1 + 2.0 ** -6
TINY = 1e-37


def lib():
    from segmented_gather_lora_amd import _build
    _build.ensure_built()
    import segmented_gather_lora_amd as sgl
    return sgl


class Case:
    def __init__(self, n, hidden, widths, rank, loras, none=0.2, bias=True, offset=0, extra=0, seed=0, ids=None,
                 stride=0):
        g = torch.Generator().manual_seed(seed * 1009 + n)
        self.n, self.hidden, self.widths, self.rank, self.loras = n, hidden, widths, rank, loras
        self.offset, self.out = offset, offset + sum(widths) + extra
        self.scale = 2.0 / math.sqrt(rank)

        def normal(*shape, sigma=1.0):
            return (torch.randn(shape, generator=g) * sigma).to(torch.bfloat16)
        if ids is None:
            ids = torch.randint(0, loras, (n,), generator=g)
            ids[torch.rand(n, generator=g) < none] = -1
        self.ids = torch.as_tensor(ids, dtype=torch.int32)
        self.stride = stride
        self.x = normal(n, hidden)
        self.w = normal(self.out, hidden, sigma=0.05)
        self.w_bias = normal(self.out, sigma=0.1) if bias else None
        self.a = [normal(loras, rank, hidden, sigma=0.05) for _ in widths]
        self.b = [normal(loras, w, rank, sigma=0.05) for w in widths]
        self.bias = [normal(loras, w, sigma=0.1) if i != 1 else None for i, w in enumerate(widths)] if bias else None
        self.dy = normal(n, self.out, sigma=0.1)


def _rows(c, m):
    return torch.nonzero(c.ids == m).flatten()


def formulas(c, x, w, w_bias, a, b, bias, dy, scale):
    """y, s, u, dx, da, db, dbias; with magnitudes in place of the values, the M(.)."""
    y = x @ w.t()
    if w_bias is not None:
        y = y + w_bias
    base, dbase = y.clone(), dy @ w
    dx = dbase.clone()
    s = [torch.zeros(c.n, c.rank, dtype=torch.float64) for _ in c.widths]
    u = [torch.zeros(c.n, c.rank, dtype=torch.float64) for _ in c.widths]
    da = [torch.zeros(t.shape, dtype=torch.float64) for t in a]
    db = [torch.zeros(t.shape, dtype=torch.float64) for t in b]
    dbias = [torch.zeros(t.shape[:2], dtype=torch.float64) for t in b]
    for m in range(c.loras):
        rows = _rows(c, m)
        if len(rows) == 0:
            continue
        col = c.offset
        for i, width in enumerate(c.widths):
            cols = slice(col, col + width)
            col += width
            si = scale * (x[rows] @ a[i][m].t())
            ui = scale * (dy[rows, cols] @ b[i][m])
            s[i][rows], u[i][rows] = si, ui
            y[rows, cols] += si @ b[i][m].t()
            if bias is not None and bias[i] is not None:
                y[rows, cols] += bias[i][m]
            dx[rows] += ui @ a[i][m]
            da[i][m] = ui.t() @ x[rows]
            db[i][m] = dy[rows, cols].t() @ si
            dbias[i][m] = dy[rows, cols].sum(0)
    return dict(y=y, s=s, u=u, dx=dx, da=da, db=db, dbias=dbias, base=base, dbase=dbase)


def reference(c):
    d = lambda t: None if t is None else [v if v is None else v.double() for v in t] if isinstance(t, list) else t.double()
    ab = lambda t: None if t is None else [v if v is None else v.double().abs() for v in t] if isinstance(t, list) else t.double().abs()
    val = formulas(c, d(c.x), d(c.w), d(c.w_bias), d(c.a), d(c.b), d(c.bias), d(c.dy), c.scale)
    mag = formulas(c, ab(c.x), ab(c.w), ab(c.w_bias), ab(c.a), ab(c.b), ab(c.bias), ab(c.dy), c.scale)
    return val, mag


def tolerances(c, val, mag):
    H, O, r, n, w = c.hidden, c.out, c.rank, c.n, max(c.widths)
    tol = {"y": U8 * val["y"].abs() + U23 * (H + 8) * mag["base"] + (U16 + U23 * (H + 2 * r + 8)) * (mag["y"] - mag["base"]),
           "dx": U8 * val["dx"].abs() + U23 * (O + 8) * mag["dbase"] + (U16 + U23 * (w + 2 * r + 8)) * (mag["dx"] - mag["dbase"]),
           "s": [U23 * (H + 8) * t for t in mag["s"]], "u": [U23 * (w + 8) * t for t in mag["u"]],
           "da": [U8 * v.abs() + (U16 + U23 * (w + 2 * n + 8)) * m for v, m in zip(val["da"], mag["da"])],
           "db": [U8 * v.abs() + (U16 + U23 * (H + 2 * n + 8)) * m for v, m in zip(val["db"], mag["db"])],
           "dbias": [U8 * v.abs() + U23 * (n + 8) * m for v, m in zip(val["dbias"], mag["dbias"])]}
    return {k: [t * SLACK + TINY for t in v] if isinstance(v, list) else v * SLACK + TINY for k, v in tol.items()}


class Run:
    """The library's buffers of a case; outputs are filled with a poison first."""

    def __init__(self, c, backward=True, poison=float("nan")):
        sgl = lib()
        dev = lambda t: None if t is None else [v if v is None else v.cuda() for v in t] if isinstance(t, list) else t.cuda()
        self.c = c

        def strided(t):   # rows further apart than their length
            if not c.stride:
                return t.cuda()
            wide = torch.full((t.shape[0], t.shape[1] + c.stride), float("nan"), dtype=t.dtype, device="cuda")
            wide[:, :t.shape[1]] = t.cuda()
            return wide[:, :t.shape[1]]
        self.x, self.w, self.dy = strided(c.x), strided(c.w), strided(c.dy)
        self.w_bias, self.a, self.b, self.bias = dev(c.w_bias), dev(c.a), dev(c.b), dev(c.bias)
        self.meta = sgl.LoraMeta(c.loras, max(c.n, 1))
        sgl.lora_prepare_meta(c.ids.cuda(), self.meta)
        S, n, r = len(c.widths), c.n, c.rank
        f = lambda shape, dt: torch.full(shape, poison, dtype=dt, device="cuda")
        self.buf, self.dbuf = f((S, n, r), torch.float32), f((S, n, r), torch.float32)
        self.y = strided(torch.full((n, c.out), poison, dtype=torch.bfloat16))
        self.dx = strided(torch.full((n, c.hidden), poison, dtype=torch.bfloat16))
        self.da = [f(t.shape, torch.bfloat16) for t in c.a]
        self.db = [f(t.shape, torch.bfloat16) for t in c.b]
        self.dbias = [f(t.shape[:2], torch.bfloat16) for t in c.b]
        self.workspace = torch.zeros(sgl.lora_linear_workspace_bytes(n, c.loras, c.hidden, c.widths, r, backward),
                                     dtype=torch.uint8, device="cuda")

    def forward(self, **kw):
        c = self.c
        lib().lora_linear(self.x, self.w, self.w_bias, self.a, self.b, self.bias, self.buf, self.y, self.meta, c.scale,
                          self.workspace, offset_start=c.offset, **kw)

    def backward(self, dx=True, dbias=True, **kw):
        c = self.c
        lib().lora_linear_backward(self.dy, self.x, self.w, self.a, self.b, self.buf, self.dbuf, self.dx if dx else None,
                                   self.da, self.db, self.dbias if dbias else None, self.meta, c.scale, self.workspace,
                                   offset_start=c.offset, **kw)

    def outputs(self):
        torch.cuda.synchronize()
        host = lambda t: [v.cpu().double() for v in t] if isinstance(t, list) else t.cpu().double()
        return {"y": host(self.y), "dx": host(self.dx), "s": list(host(self.buf)), "u": list(host(self.dbuf)),
                "da": host(self.da), "db": host(self.db), "dbias": host(self.dbias)}


def check(c, got, keys=("y", "dx", "s", "u", "da", "db", "dbias")):
    val, mag = reference(c)
    tol = tolerances(c, val, mag)
    on = c.ids >= 0
    for k in keys:
        many = isinstance(val[k], list)
        for i, (g, v, t) in enumerate(zip(got[k] if many else [got[k]], val[k] if many else [val[k]],
                                          tol[k] if many else [tol[k]])):
            if k in ("s", "u"):   # rows of tokens without an adapter are not touched
                assert torch.isnan(g[~on]).all(), "%s[%d]: rows without an adapter" % (k, i)
                g, v, t = g[on], v[on], t[on]
            assert torch.isfinite(g).all(), "%s[%d] has values that are not finite" % (k, i)
            worst = ((g - v).abs() / t).max().item() if g.numel() else 0.0
            assert worst <= 1, "%s[%d]: %.3g times the tolerance" % (k, i, worst)


CASES = {
    "one token": dict(n=1, hidden=72, widths=[40, 16], rank=8, loras=3, none=0.0),
    "one token without adapter": dict(n=1, hidden=64, widths=[64], rank=16, loras=2, none=1.0),
    "smallest": dict(n=2, hidden=8, widths=[8], rank=8, loras=1),
    "few tokens, long K": dict(n=17, hidden=1032, widths=[264, 8, 136], rank=24, loras=9),
    "32": dict(n=32, hidden=520, widths=[136], rank=16, loras=32, none=0.0),
    "33": dict(n=33, hidden=264, widths=[72, 72], rank=40, loras=5, extra=24, offset=16),
    "129": dict(n=129, hidden=136, widths=[200, 8], rank=128, loras=4, stride=8),
    "one adapter": dict(n=257, hidden=264, widths=[320], rank=64, loras=1, none=0.0),
    "many adapters": dict(n=300, hidden=200, widths=[152], rank=8, loras=290),
    "most adapters": dict(n=70, hidden=72, widths=[72], rank=8, loras=1023),
    "eight slices": dict(n=45, hidden=72, widths=[8, 16, 24, 32, 40, 8, 16, 24], rank=32, loras=3),
    "no adapter at all": dict(n=150, hidden=136, widths=[72], rank=16, loras=4, none=1.0),
    "long K split": dict(n=200, hidden=4104, widths=[264], rank=16, loras=6, bias=False),
    "wide output": dict(n=40, hidden=72, widths=[4104, 72], rank=72, loras=3),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(CASES))
def test_against_formulas(name):
    c = Case(**CASES[name])
    r = Run(c)
    r.forward()
    r.backward()
    check(c, r.outputs())
    # the workspace's counters are zero again, and a second pass gives the same
    # bits (db reads buf, whose last bits may vary where the shrink splits K)
    first = r.outputs()
    r.forward()
    r.backward()
    again = r.outputs()
    assert torch.equal(first["dx"], again["dx"])
    for k in ("da", "dbias"):
        for p, q in zip(first[k], again[k]):
            assert torch.equal(p, q), k


@pytest.mark.gpu
@pytest.mark.parametrize("hidden,widths,keys", [
    (72, [2568, 512], ("y", "s")),                        # forward: 17 x 13 tiles of 256 x 256
    (3080, [64, 8], ("dx", "da", "db", "dbias", "u"))])   # backward: likewise
def test_large_tiles(hidden, widths, keys):
    c = Case(n=4097, hidden=hidden, widths=widths, rank=40, loras=37)
    r = Run(c)
    r.forward()
    r.backward()
    check(c, r.outputs(), keys)


@pytest.mark.gpu
def test_empty_batch():
    c = Case(n=0, hidden=64, widths=[64, 8], rank=8, loras=3)
    r = Run(c)
    r.forward()
    r.backward()
    got = r.outputs()
    for k in ("da", "db", "dbias"):
        assert all((t == 0).all() for t in got[k]), k


@pytest.mark.gpu
def test_optional_results():
    c = Case(n=50, hidden=72, widths=[72], rank=8, loras=3)
    r = Run(c)
    r.forward()
    r.backward(dx=False, dbias=False)
    got = r.outputs()
    check(c, got, ("y", "da", "db"))
    assert torch.isnan(got["dx"]).all() and all(torch.isnan(t).all() for t in got["dbias"])


@pytest.mark.gpu
def test_ids_out_of_range_count_as_none():
    ids = [0, 5, -2, 1, 1, 2, 77, -1]
    c = Case(n=8, hidden=72, widths=[72], rank=8, loras=3, ids=ids)
    r = Run(c)
    r.forward()
    r.backward()
    got = r.outputs()
    assert int(r.meta.views()["status"].item()) == lib().LORA_ERR_ID_RANGE
    c.ids = torch.tensor([i if 0 <= i < 3 else -1 for i in ids], dtype=torch.int32)
    check(c, got)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [48, 300])
def test_not_finite_stays_where_it_belongs(n):
    """A diverged adapter, an infinite activation: other tokens and other
    adapters' gradients keep their exact results."""
    c = Case(n=n, hidden=136, widths=[136, 40], rank=16, loras=5)
    r = Run(c)
    r.forward()
    r.backward()
    clean = r.outputs()
    bad = int(torch.nonzero(c.ids == 3)[0])
    r.b[0][2] = float("nan")
    r.a[1][2] = float("inf")
    r.bias[0][2] = float("nan")
    r.x[bad, 5] = float("inf")
    r.dy[bad, 7] = float("nan")
    r.forward()
    r.backward()
    got = r.outputs()
    rows = (c.ids != 2) & (torch.arange(n) != bad)
    assert torch.equal(got["y"][rows], clean["y"][rows]) and torch.equal(got["dx"][rows], clean["dx"][rows])
    for m in (0, 1, 4):
        for k in ("da", "db", "dbias"):
            for p, q in zip(got[k], clean[k]):
                assert torch.equal(p[m], q[m]), (k, m)
    assert not torch.isfinite(got["y"][c.ids == 2]).all() and not torch.isfinite(got["y"][bad]).all()


@pytest.mark.gpu
def test_gradients_against_differences():
    """<gradient, direction> against central differences of sum(dy * y), y in
    64 bits (the sum is linear in x and w_bias and bilinear in the adapters, so
    the differences are exact up to 64-bit rounding)."""
    c = Case(n=90, hidden=136, widths=[72, 40], rank=16, loras=4)
    r = Run(c)
    r.forward()
    r.backward()
    got = r.outputs()
    val, mag = reference(c)
    tol = tolerances(c, val, mag)
    g = torch.Generator().manual_seed(5)
    d = lambda t: None if t is None else [v if v is None else v.double() for v in t] if isinstance(t, list) else t.double()

    def loss(x, a, b, bias):
        return (formulas(c, x, d(c.w), d(c.w_bias), a, b, bias, d(c.dy), c.scale)["y"] * d(c.dy)).sum().item()
    base = dict(x=d(c.x), a=d(c.a), b=d(c.b), bias=d(c.bias))
    for key, out in (("x", "dx"), ("a", "da"), ("b", "db"), ("bias", "dbias")):
        for i in range(1 if key == "x" else len(c.widths)):
            at = base[key] if key == "x" else base[key][i]
            if at is None:
                continue
            step = torch.randn(at.shape, generator=g, dtype=torch.float64)
            vals = []
            for sign in (1, -1):
                moved = dict(base)
                if key == "x":
                    moved[key] = at + sign * 1e-3 * step
                else:
                    moved[key] = [at + sign * 1e-3 * step if j == i else t for j, t in enumerate(base[key])]
                vals.append(loss(**moved))
            grad = got[out] if key == "x" else got[out][i]
            bound = tol[out] if key == "x" else tol[out][i]
            diff = (vals[0] - vals[1]) / 2e-3
            assert abs((grad * step).sum().item() - diff) <= (bound * step.abs()).sum().item() + 1e-7 * abs(diff)


@pytest.mark.gpu
def test_other_stream_and_graph_replays():
    """The calls on a side stream, and captured: every replay equals the eager results."""
    c = Case(n=70, hidden=1032, widths=[136, 72], rank=16, loras=6)
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
    for k, v in r.outputs().items():
        assert all(torch.equal(torch.nan_to_num(p), torch.nan_to_num(q)) for p, q in zip(v, eager[k])) or k in ("s", "y", "db")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r.forward()
        r.backward()
    for _ in range(4):
        for t in [r.y, r.dx] + r.da + r.db + r.dbias:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        check(c, r.outputs())
        r.x.mul_(1.0)   # eager work between the replays


# ------------------------------------------------------------------ refusals (no GPU)

def _fake(sgl, n):
    base = 0x7f0000000000
    m = sgl.lora_meta_bind(base, sgl.lora_meta_bytes(4, 128), 4, 128)
    m.num_tokens = n
    return m


def _ptrs(*v):
    return (ctypes.c_void_p * len(v))(*v)


def test_workspace_sizes():
    sgl = lib()
    small = sgl.lora_linear_workspace_bytes(16, 4, 64, [64, 32], 8)
    assert 0 < small <= sgl.lora_linear_workspace_bytes(16, 4, 64, [64, 32], 8, True)
    L = sgl.lib
    W = (ctypes.c_int * 2)(64, 32)
    for bad in ((-1, 4, 64, W, 2, 8), (16, 0, 64, W, 2, 8), (16, 1024, 64, W, 2, 8), (16, 4, 60, W, 2, 8),
                (16, 4, 64, W, 0, 8), (16, 4, 64, W, 9, 8), (16, 4, 64, None, 2, 8), (16, 4, 64, W, 2, 12),
                (16, 4, 64, (ctypes.c_int * 2)(64, 12), 2, 8)):
        assert L.lora_linear_workspace_bytes(*bad, 0) == 0
    with pytest.raises(sgl.LoraError):
        sgl.lora_linear_workspace_bytes(16, 4, 60, [64], 8)


def test_linear_refusals():
    sgl = lib()
    L, m = sgl.lib, _fake(sgl, 32)
    need = sgl.lora_linear_workspace_bytes(32, 4, 64, [64, 32], 16)
    ok = dict(x=0x10000, ldx=64, n=32, h=64, w=0x20000, ldw=64, out=96, wb=0x30000, a=_ptrs(0x40000, 0x50000),
              b=_ptrs(0x60000, 0x70000), bias=None, wd=(ctypes.c_int * 2)(64, 32), s=2, r=16, buf=0x80000, y=0x90000,
              ldy=96, off=0, ws=0xa0000, nb=need, meta=m)

    def call(**kw):
        v = dict(ok, **kw)
        return L.lora_linear(v["x"], v["ldx"], v["n"], v["h"], v["w"], v["ldw"], v["out"], v["wb"], v["a"], v["b"],
                             v["bias"], v["wd"], v["s"], v["r"], v["buf"], v["y"], v["ldy"], v["off"],
                             ctypes.byref(v["meta"]), 1.0, v["ws"], v["nb"], None)
    E = sgl
    assert call(n=31) == E.LORA_ERR_NUM_TOKENS and call(meta=_fake(sgl, -1)) == E.LORA_ERR_NUM_TOKENS
    assert call(s=0) == E.LORA_ERR_SLICES and call(s=9) == E.LORA_ERR_SLICES
    for kw in (dict(h=60), dict(ldx=56), dict(ldw=56), dict(ldw=68), dict(r=12), dict(r=136), dict(out=92),
               dict(out=88), dict(ldy=88), dict(off=8), dict(off=-8), dict(wd=(ctypes.c_int * 2)(64, 12))):
        assert call(**kw) == E.LORA_ERR_SHAPE, kw
    for kw in (dict(x=None), dict(w=None), dict(buf=None), dict(y=None), dict(a=None), dict(b=None), dict(wd=None),
               dict(ws=None), dict(a=_ptrs(0x40000, None)), dict(b=_ptrs(None, 0x70000))):
        assert call(**kw) == E.LORA_ERR_NULL, kw
    for kw in (dict(x=0x10008), dict(w=0x20008), dict(wb=0x30002), dict(a=_ptrs(0x40000, 0x50008)),
               dict(b=_ptrs(0x60002, 0x70000)), dict(bias=_ptrs(None, 0x70008)), dict(buf=0x80004), dict(y=0x90008)):
        assert call(**kw) == E.LORA_ERR_ALIGN, kw
    assert call(ws=0xa0010) == E.LORA_ERR_BUFFER and call(nb=256) == E.LORA_ERR_BUFFER
    assert call(n=0, meta=_fake(sgl, 0)) == E.LORA_OK


def test_linear_backward_refusals():
    sgl = lib()
    L, m = sgl.lib, _fake(sgl, 32)
    need = sgl.lora_linear_workspace_bytes(32, 4, 64, [64, 32], 16, True)
    two = _ptrs(0x110000, 0x120000)
    ok = dict(dy=0x90000, lddy=96, x=0x10000, ldx=64, n=32, h=64, w=0x20000, ldw=64, out=96, a=_ptrs(0x40000, 0x50000),
              b=_ptrs(0x60000, 0x70000), wd=(ctypes.c_int * 2)(64, 32), s=2, r=16, buf=0x80000, dbuf=0x88000,
              dx=0xb0000, lddx=64, da=two, db=two, dbias=None, off=0, ws=0xa0000, nb=need, meta=m)

    def call(**kw):
        v = dict(ok, **kw)
        return L.lora_linear_backward(v["dy"], v["lddy"], v["x"], v["ldx"], v["n"], v["h"], v["w"], v["ldw"], v["out"],
                                      v["a"], v["b"], v["wd"], v["s"], v["r"], v["buf"], v["dbuf"], v["dx"], v["lddx"],
                                      v["da"], v["db"], v["dbias"], v["off"], ctypes.byref(v["meta"]), 1.0, v["ws"],
                                      v["nb"], None)
    E = sgl
    assert call(n=31) == E.LORA_ERR_NUM_TOKENS and call(s=9) == E.LORA_ERR_SLICES
    for kw in (dict(h=60), dict(lddy=88), dict(lddx=56), dict(lddx=68), dict(out=88), dict(r=12), dict(off=8)):
        assert call(**kw) == E.LORA_ERR_SHAPE, kw
    for kw in (dict(dy=None), dict(x=None), dict(buf=None), dict(dbuf=None), dict(da=None), dict(db=None),
               dict(da=_ptrs(0x110000, None)), dict(w=None), dict(ws=None)):
        assert call(**kw) == E.LORA_ERR_NULL, kw
    for kw in (dict(dy=0x90008), dict(dbuf=0x88004), dict(dx=0xb0008), dict(da=_ptrs(0x110008, 0x120000)),
               dict(dbias=_ptrs(None, 0x70002))):
        assert call(**kw) == E.LORA_ERR_ALIGN, kw
    assert call(nb=need // 2) == E.LORA_ERR_BUFFER


def test_binding_refuses_what_the_library_cannot_see():
    """Host tensors and wrong types raise before the library is called (no GPU needed)."""
    sgl = lib()

    class Meta:
        num_tokens, max_loras, max_num_tokens = 4, 2, 4
        region = torch.zeros(1, dtype=torch.uint8)
    x = torch.zeros(4, 16, dtype=torch.bfloat16)
    w = torch.zeros(8, 16, dtype=torch.bfloat16)
    a, b = [torch.zeros(2, 8, 16, dtype=torch.bfloat16)], [torch.zeros(2, 8, 8, dtype=torch.bfloat16)]
    buf, y = torch.zeros(1, 4, 8), torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        sgl.lora_linear(x, w, None, a, b, None, buf, y, Meta(), 1.0, torch.zeros(8, dtype=torch.uint8))
    with pytest.raises(sgl.LoraError):
        sgl.lora_linear(x[:3], w, None, a, b, None, buf, y, Meta(), 1.0, torch.zeros(8, dtype=torch.uint8))
