"""Microscaled 4-bit numbers and the shared projection held in them, against the
formulas in 64 bits on the CPU.

Quantization and its inverse are exact: every code, scale and number has to be
equal.  The projection's tolerances are those of test_linear.py with the numbers
that the codes stand for as its matrix (a product of two such numbers is exact in
float32, so that quantized activations add nothing to them): its sums are float32
over the same number of products, and results are rounded once.
"""
import ctypes
import math
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(__file__))
import test_linear  # noqa: E402
from test_linear import Case, lib  # noqa: E402

GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


# ---------------------------------------------------------------- the format, in 64 bits

def quantized(x):
    """codes and scale bytes of rows of x (float64 on the CPU), by the format's
    definition, and the numbers that they stand for."""
    n, k = x.shape
    blocks = (k + 31) // 32
    codes = torch.zeros((n, blocks * 32), dtype=torch.int64)
    scales = torch.zeros((n, (blocks + 3) // 4 * 4), dtype=torch.int64)
    held = torch.zeros((n, k), dtype=torch.float64)
    for b in range(blocks):
        part = x[:, 32 * b:32 * b + 32]
        top = part.abs().amax(1)
        finite = torch.isfinite(part).all(1)
        safe = torch.where(finite & (top > 0), top, torch.ones_like(top))
        power = torch.where(finite & (top > 0), torch.frexp(safe)[1].double() - 3, torch.full_like(top, -127.0)).clamp(min=-127)
        m = torch.where(finite[:, None], part, torch.zeros_like(part)).abs() / torch.exp2(power)[:, None]
        dist = (m[..., None] - GRID).abs()
        best = dist.amin(-1, keepdim=True)
        # of two that are equally near, the one of even code
        near = torch.where(dist == best, torch.arange(8) + 8 * (torch.arange(8) % 2), 99).amin(-1) % 8
        sign = torch.signbit(part) & finite[:, None]
        codes[:, 32 * b:32 * b + part.shape[1]] = near + 8 * sign
        scales[:, b] = torch.where(finite, power + 127, torch.full_like(power, 255.0)).long()
        value = torch.where(sign, -GRID[near], GRID[near]) * torch.exp2(power)[:, None]
        held[:, 32 * b:32 * b + part.shape[1]] = torch.where(finite[:, None], value, torch.full_like(value, float("nan")))
    return (codes[:, ::2] | codes[:, 1::2] << 4).to(torch.uint8), scales.to(torch.uint8), held


def numbers(kind, n, k, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, k), generator=g, dtype=torch.float64)
    if kind == "rows":            # rows of very different sizes
        x *= torch.exp2(60 * torch.randn((n, 1), generator=g, dtype=torch.float64)).clamp(2.0 ** -130, 2.0 ** 120)
    elif kind == "borders":       # midpoints, powers, zeros and what is next to them
        pick = torch.tensor([0, 0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 6.5, 7, 7.5, 7.9375], dtype=torch.float64)
        x = pick[torch.randint(0, len(pick), (n, k), generator=g)] * torch.sign(x) * torch.exp2(
            torch.randint(-20, 20, (n, 1), generator=g).double())
        x = x * (1 + torch.randint(-1, 2, (n, k), generator=g).double() * torch.finfo(dtype).eps)
    elif kind == "tiny":          # down to subnormal numbers
        x *= 2.0 ** torch.randint(-149, -118, (n, 1), generator=g).double()
    elif kind == "zeros":
        x[torch.rand((n, k), generator=g) < 0.9] = 0
        x[n // 2:] = 0
    elif kind == "not finite":
        x[torch.rand((n, k), generator=g) < 0.02] = float("inf")
        x[torch.rand((n, k), generator=g) < 0.02] = float("nan")
    elif kind == "largest":
        x = torch.sign(x) * torch.finfo(dtype).max * torch.rand((n, k), generator=g, dtype=torch.float64)
    return x.to(dtype)


def rows_apart(t, extra, fill):
    """t on the GPU with `extra` more columns behind each row."""
    wide = torch.full((t.shape[0], t.shape[1] + extra), fill, dtype=t.dtype, device="cuda")
    wide[:, :t.shape[1]] = t.cuda()
    return wide, wide[:, :t.shape[1]]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["normal", "rows", "borders", "tiny", "zeros", "not finite", "largest"])
@pytest.mark.parametrize("n,k", [(1, 8), (3, 32), (37, 136), (65, 1032), (5, 4104)])
def test_quantize(dtype, kind, n, k):
    sgl = lib()
    x = numbers(kind, n, k, 7 * n + k, dtype)
    codes, scales, held = quantized(x.double())
    code_bytes, scale_bytes = sgl.lora_mx_row_bytes(k)
    assert (code_bytes, scale_bytes) == (codes.shape[1], scales.shape[1])
    all_x, gx = rows_apart(x, 8, float("nan"))
    all_c, gc = rows_apart(torch.full((n, code_bytes), 0xAA, dtype=torch.uint8), 16, 0x55)
    all_s, gs = rows_apart(torch.full((n, scale_bytes), 0xAA, dtype=torch.uint8), 4, 0x55)
    sgl.lora_mx_quantize(gx, gc, gs)
    assert torch.equal(gs.cpu(), scales)
    assert torch.equal(gc.cpu(), codes)
    assert (all_c[:, code_bytes:] == 0x55).all() and (all_s[:, scale_bytes:] == 0x55).all()
    for to in (torch.bfloat16, torch.float32):
        all_o, out = rows_apart(torch.full((n, k), 7.0, dtype=to), 8, 7.0)
        sgl.lora_mx_dequantize(gc, gs, out)
        want = held.to(to)
        got = out.cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(got, nan=1.0), torch.nan_to_num(want, nan=1.0))
        assert (all_o[:, k:] == 7.0).all()


@pytest.mark.gpu
def test_dequantize_every_code_and_scale():
    sgl = lib()
    codes = (torch.arange(256 * 16) % 256).reshape(256, 16).to(torch.uint8)
    scales = torch.zeros((256, 4), dtype=torch.uint8)
    scales[:, 0] = torch.arange(256)
    scales[:, 1:] = 255                       # of no block: not used
    for to in (torch.bfloat16, torch.float32):
        out = torch.empty((256, 32), dtype=to, device="cuda")
        sgl.lora_mx_dequantize(codes.cuda(), scales.cuda(), out)
        both = torch.stack((codes & 15, codes >> 4), 2).flatten(1).long()
        value = torch.cat((GRID, -GRID))[both] * torch.exp2(torch.arange(256).double() - 127)[:, None]
        value[255] = float("nan")
        want = value.to(to)
        assert torch.equal(torch.nan_to_num(out.cpu(), nan=1.0), torch.nan_to_num(want, nan=1.0))


@pytest.mark.gpu
def test_quantize_no_rows_and_large_offsets():
    sgl = lib()
    empty = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    none = torch.empty((0, 32), dtype=torch.uint8, device="cuda"), torch.empty((0, 4), dtype=torch.uint8, device="cuda")
    sgl.lora_mx_quantize(empty, *none)
    # more than 2^32 bytes and 2^31 numbers from the first row to the last
    n, k = 70000, 32776
    x = torch.empty((n, k), dtype=torch.bfloat16, device="cuda").fill_(1.0)
    g = torch.Generator(device="cuda").manual_seed(3)
    x[-3:] = torch.randn((3, k), generator=g, device="cuda").to(torch.bfloat16)
    code_bytes, scale_bytes = sgl.lora_mx_row_bytes(k)
    codes = torch.zeros((n, code_bytes), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((n, scale_bytes), dtype=torch.uint8, device="cuda")
    sgl.lora_mx_quantize(x, codes, scales)
    want = quantized(x[-3:].cpu().double())
    assert torch.equal(codes[-3:].cpu(), want[0]) and torch.equal(scales[-3:].cpu(), want[1])
    first = quantized(x[:1].cpu().double())
    assert (codes[:-3] == first[0].cuda()).all() and (scales[:-3] == first[1].cuda()).all()
    sgl.lora_mx_dequantize(codes, scales, x)
    assert torch.equal(x[-3:].cpu(), want[2].to(torch.bfloat16)) and (x[:-3] == 1).all()


# ---------------------------------------------------------------- the projection

class MxCase(Case):
    """A case of lora_linear whose matrix is what codes stand for."""

    def __init__(self, acts="bf16", **kw):
        super().__init__(**kw)
        self.codes, self.scales, self.w = quantized(self.w.double())
        self.acts = acts
        self.seen = self.x.double() if acts == "bf16" else quantized(self.x.double())[2]

    def reference(self):
        """test_linear's values and magnitudes; W's product reads what the call sees of x."""
        val, mag = test_linear.reference(self)
        w = self.w
        val["y"] = val["y"] + (self.seen - self.x.double()) @ w.t()
        change = (self.seen.abs() - self.x.double().abs()) @ w.abs().t()
        mag["y"], mag["base"] = mag["y"] + change, mag["base"] + change
        return val, mag


class MxRun(test_linear.Run):
    def __init__(self, c, backward=True, pad=0, **kw):
        super().__init__(c, backward, **kw)
        sgl = lib()
        # the rows' padding, and what the last block and dword hold past them, is not used
        self.codes = rows_apart(c.codes, pad, 0x77)[1]
        self.scales = rows_apart(c.scales, pad, 255)[1]
        k = c.hidden
        if k % 32:
            self.codes[:, k // 2:] = 0x5B
        blocks = (k + 31) // 32
        self.scales[:, blocks:] = 255
        self.workspace = torch.full(
            (sgl.lora_linear_mx_workspace_bytes(c.n, c.loras, c.hidden, c.out, c.widths, c.rank, backward),), 0xFF,
            dtype=torch.uint8, device="cuda")

    def forward(self, **kw):
        c = self.c
        lib().lora_linear_mx(self.x, self.codes, self.scales, self.w_bias, self.a, self.b, self.bias, self.buf, self.y,
                             self.meta, c.scale, self.workspace, offset_start=c.offset, quantize_x=c.acts == "mxfp4", **kw)

    def backward(self, dx=True, dbias=True, **kw):
        c = self.c
        lib().lora_linear_mx_backward(self.dy, self.x, self.codes, self.scales, self.a, self.b, self.buf, self.dbuf,
                                      self.dx if dx else None, self.da, self.db, self.dbias if dbias else None, self.meta,
                                      c.scale, self.workspace, offset_start=c.offset, **kw)


def check(c, got, keys=("y", "dx", "s", "u", "da", "db", "dbias")):
    val, mag = c.reference()
    tol = test_linear.tolerances(c, val, mag)
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


CASES = dict(test_linear.CASES)
CASES.update({
    "block of 8": dict(n=40, hidden=40, widths=[72], rank=8, loras=3),
    "blocks of 24": dict(n=20, hidden=88, widths=[72, 264], rank=16, loras=3),
    "tile of few rows": dict(n=130, hidden=2056, widths=[520, 24], rank=16, loras=7, extra=8, stride=24),
    "a span and a block": dict(n=70, hidden=288, widths=[136], rank=16, loras=4),
    "wide, short K": dict(n=300, hidden=24, widths=[1032], rank=24, loras=4),
})


@pytest.mark.gpu
@pytest.mark.parametrize("acts", ["bf16", "mxfp4"])
@pytest.mark.parametrize("name", list(CASES))
def test_against_formulas(name, acts):
    c = MxCase(acts=acts, **CASES[name])
    r = MxRun(c, pad=0 if c.stride == 0 else 48)
    r.forward()
    r.backward()
    first = r.outputs()
    check(c, first)
    r.workspace.fill_(0x7F)
    r.forward()
    r.backward()
    again = r.outputs()
    assert torch.equal(first["dx"], again["dx"])
    for k in ("da", "dbias"):
        for p, q in zip(first[k], again[k]):
            assert torch.equal(p, q), k


@pytest.mark.gpu
@pytest.mark.parametrize("acts,n,hidden,widths,keys", [
    ("bf16", 4097, 72, [2568, 512], ("y", "s")),              # 256 x 256 tiles, one K step and a rest
    ("bf16", 4097, 328, [2568, 512], ("y", "s")),             # a pinned loop of few steps
    ("bf16", 1100, 1032, [5128, 5120], ("y", "s")),
    ("mxfp4", 4097, 72, [2568, 512], ("y", "s")),
    ("mxfp4", 1100, 1032, [5128, 5120], ("y", "s")),
    ("mxfp4", 1100, 2088, [5128, 5120], ("y", "s")),
    ("bf16", 520, 264, [6144], ("y", "s")),                   # 128 x 128 tiles
    ("bf16", 520, 520, [6152], ("y", "s")),
    ("mxfp4", 520, 520, [6152], ("y", "s")),
    ("mxfp4", 520, 1544, [6152], ("y", "s")),
    ("bf16", 4097, 3080, [64, 8], ("dx", "da", "db", "dbias", "u")),   # backward: 256 x 256
    ("bf16", 4097, 3080, [328, 8], ("dx", "da", "db", "dbias", "u")),
    ("bf16", 520, 6152, [264, 8], ("dx", "da", "db", "dbias", "u"))])
def test_large_tiles(acts, n, hidden, widths, keys):
    c = MxCase(acts=acts, n=n, hidden=hidden, widths=widths, rank=40, loras=37)
    r = MxRun(c)
    r.forward()
    r.backward()
    check(c, r.outputs(), keys)


@pytest.mark.gpu
@pytest.mark.parametrize("acts,n,hidden,out", [
    ("mxfp4", 520, 768, 6144),       # whole steps of 256 and no rest: three of them, four, five
    ("mxfp4", 520, 1024, 6144),
    ("mxfp4", 300, 1280, 264),       # small tiles
    ("mxfp4", 129, 512, 264),
    ("bf16", 40, 8328, 72),          # 66 steps of 128: the scales' two buffers, each twice
    ("bf16", 70, 4096, 136),         # 32 steps
    ("bf16", 33, 384, 64),
    ("bf16", 100, 128, 200)])
def test_whole_steps(acts, n, hidden, out):
    for rank, none in ((8, 0.2), (40, 0.0)):
        c = MxCase(acts=acts, n=n, hidden=hidden, widths=[out], rank=rank, loras=2, none=none, seed=rank)
        r = MxRun(c)
        r.forward()
        check(c, r.outputs(), ("y", "s"))


@pytest.mark.gpu
@pytest.mark.parametrize("acts", ["bf16", "mxfp4"])
@pytest.mark.parametrize("n", [128, 300])
def test_one_adapter_has_whole_tiles(acts, n):
    """One adapter for all tokens, ranks of one and of several blocks, slices that end
    inside a tile; and adapters that change at a tile's edge."""
    for rank in (16, 32, 72):
        for ids in ([0] * n, [i // 128 for i in range(n)], [1] * 100 + [0] * (n - 100)):
            c = MxCase(acts=acts, n=n, hidden=264, widths=[5000, 72, 10000], rank=rank, loras=3, ids=ids, extra=16)
            r = MxRun(c, backward=False)
            r.forward()
            check(c, r.outputs(), ("y", "s"))


@pytest.mark.gpu
@pytest.mark.parametrize("acts", ["bf16", "mxfp4"])
def test_biases_of_few_and_of_many_adapters(acts):
    for loras, seed in ((2, 0), (4, 1), (5, 2), (40, 3)):
        for bias in (True, False):
            c = MxCase(acts=acts, n=200, hidden=136, widths=[136, 40, 24], rank=8, loras=loras, seed=seed, bias=bias)
            if not bias:      # the projection's alone
                c.w_bias = torch.randn(c.out, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)
            r = MxRun(c, backward=False)
            r.forward()
            check(c, r.outputs(), ("y", "s"))


@pytest.mark.gpu
@pytest.mark.parametrize("acts", ["bf16", "mxfp4"])
def test_powers_from_the_smallest_to_the_largest(acts):
    """Scale bytes over their whole range, where the sums stay in range."""
    for n in (5, 40, 300):
        c = MxCase(acts=acts, n=n, hidden=264, widths=[136], rank=8, loras=2, none=1.0, bias=False)
        span = torch.randint(0, 60, (c.out, 1)) * 4          # a power a column of y: 2^-127 .. 2^109
        c.scales[:, :9] = (span + torch.randint(0, 4, (c.out, 9))).to(torch.uint8)
        both = torch.stack((c.codes & 15, c.codes >> 4), 2).flatten(1).long()
        held = torch.cat((GRID, -GRID))[both] * torch.exp2(c.scales[:, :9].double() - 127).repeat_interleave(32, 1)
        c.w = held[:, :264].contiguous()
        r = MxRun(c)
        r.forward()
        got = r.outputs()["y"]
        base, mag = c.seen @ c.w.t(), c.seen.abs() @ c.w.abs().t()
        # beside test_linear's bound: products and sums below 2^-126 may be cut to 0, each 2^-126
        tol = (2.0 ** -8 * base.abs() + 2.0 ** -23 * (264 + 8) * mag) * (1 + 2.0 ** -6) + 2.0 ** -126 * (264 + 8)
        assert ((got - base).abs() <= tol).all()


@pytest.mark.gpu
@pytest.mark.parametrize("acts", ["bf16", "mxfp4"])
@pytest.mark.parametrize("n", [1, 30, 48, 300])
def test_not_finite_stays_where_it_belongs(n, acts):
    c = MxCase(acts=acts, n=n, hidden=136, widths=[136, 40], rank=16, loras=5, none=0.3)
    r = MxRun(c)
    r.forward()
    r.backward()
    clean = r.outputs()
    column, bad = 17, n // 2
    r.scales[column, 1] = 255                 # a block of the matrix that is not a number
    r.x[bad, 133] = float("inf")
    r.dy[bad, 7] = float("nan")
    r.forward()
    r.backward()
    got = r.outputs()
    rows = torch.arange(n) != bad
    cols = torch.arange(c.out) != column
    assert torch.equal(got["y"][rows][:, cols], clean["y"][rows][:, cols])
    assert torch.isnan(got["y"][:, column]).all()
    assert not torch.isfinite(got["y"][bad]).any() if acts == "mxfp4" else not torch.isfinite(got["y"][bad]).all()
    hidden = (torch.arange(c.hidden) < 32) | (torch.arange(c.hidden) >= 64)
    assert torch.equal(got["dx"][rows][:, hidden], clean["dx"][rows][:, hidden])
    assert torch.isnan(got["dx"][:, ~hidden]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("acts", ["bf16", "mxfp4"])
def test_empty_batch(acts):
    c = MxCase(acts=acts, n=0, hidden=64, widths=[64, 8], rank=8, loras=3)
    r = MxRun(c)
    r.forward()
    r.backward()
    got = r.outputs()
    for k in ("da", "db", "dbias"):
        assert all((t == 0).all() for t in got[k]), k


@pytest.mark.gpu
@pytest.mark.parametrize("acts", ["bf16", "mxfp4"])
@pytest.mark.parametrize("n", [7, 90, 600])
def test_replays_on_another_stream(n, acts):
    """A captured step on a stream of its own, replayed over other inputs, with
    eager work between the replays."""
    c = MxCase(acts=acts, n=n, hidden=264, widths=[520, 72], rank=16, loras=6)
    r = MxRun(c)
    other = MxCase(acts=acts, n=n, hidden=264, widths=[520, 72], rank=16, loras=6, seed=1, ids=c.ids)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        r.forward()
        r.backward()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        r.forward()
        r.backward()
    for k in range(4):
        now = other if k % 2 else c
        for name in ("x", "dy", "codes", "scales"):
            getattr(r, name)[:, :getattr(now, name).shape[1]].copy_(getattr(now, name))
        for t in [r.y, r.dx] + r.da + r.db:
            t.fill_(float("nan"))
        r.workspace.fill_(0xFF)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        kept = {k: getattr(c, k) for k in ("x", "dy", "codes", "scales", "w", "seen")}
        for name in kept:
            setattr(c, name, getattr(now, name))
        check(c, r.outputs(), ("y", "dx", "da", "db"))
        for name, v in kept.items():
            setattr(c, name, v)


@pytest.mark.gpu
def test_a_large_workspace_serves_small_batches():
    sgl = lib()
    sizes = [sgl.lora_linear_mx_workspace_bytes(n, 5, 264, 136, [136], 16, True) for n in range(0, 2000, 37)]
    assert sizes == sorted(sizes)
    for acts in ("bf16", "mxfp4"):
        c = MxCase(acts=acts, n=70, hidden=264, widths=[136], rank=16, loras=5)
        r = MxRun(c)
        r.workspace = torch.full((sizes[-1],), 0xFF, dtype=torch.uint8, device="cuda")
        r.forward()
        r.backward()
        check(c, r.outputs())


# ---------------------------------------------------------------- refusals

def _fake_meta(sgl, n):
    m = sgl.lora_meta_bind(0x7f0000000000, sgl.lora_meta_bytes(4, 128), 4, 128)
    m.num_tokens = n
    return m


def test_refusals_of_the_conversions():
    sgl = lib()
    L = sgl.lib
    ok = dict(x=0x10000, type=sgl.LORA_BF16, ldx=72, rows=5, cols=72, codes=0x20000, ldc=48, scales=0x30000, lds=4)

    def to(**kw):
        a = dict(ok, **kw)
        return L.lora_mx_quantize(a["x"], a["type"], a["ldx"], a["rows"], a["cols"], a["codes"], a["ldc"], a["scales"],
                                  a["lds"], None)

    def back(**kw):
        a = dict(ok, **kw)
        return L.lora_mx_dequantize(a["codes"], a["ldc"], a["scales"], a["lds"], a["rows"], a["cols"], a["x"], a["type"],
                                    a["ldx"], None)
    for call in (to, back):
        assert call(type=2) == sgl.LORA_ERR_SHAPE and call(type=-1) == sgl.LORA_ERR_SHAPE
        assert call(cols=0) == sgl.LORA_ERR_SHAPE and call(cols=70) == sgl.LORA_ERR_SHAPE
        assert call(cols=16777224, ldx=16777224, ldc=1 << 24, lds=1 << 20) == sgl.LORA_ERR_SHAPE
        assert call(ldx=64) == sgl.LORA_ERR_SHAPE and call(ldx=76) == sgl.LORA_ERR_SHAPE
        assert call(ldc=32) == sgl.LORA_ERR_SHAPE and call(ldc=56) == sgl.LORA_ERR_SHAPE
        assert call(lds=0) == sgl.LORA_ERR_SHAPE and call(lds=6) == sgl.LORA_ERR_SHAPE
        assert call(rows=-1) == sgl.LORA_ERR_SHAPE and call(rows=1 << 31) == sgl.LORA_ERR_SHAPE
        assert call(x=None) == sgl.LORA_ERR_NULL and call(codes=None) == sgl.LORA_ERR_NULL
        assert call(scales=None) == sgl.LORA_ERR_NULL
        assert call(x=0x10008) == sgl.LORA_ERR_ALIGN and call(codes=0x20008) == sgl.LORA_ERR_ALIGN
        assert call(scales=0x30002) == sgl.LORA_ERR_ALIGN
        assert call(rows=0) == sgl.LORA_OK and call(rows=0, x=None, codes=None, scales=None) == sgl.LORA_OK


def test_refusals_of_the_projection():
    sgl = lib()
    L = sgl.lib
    P = lambda *v: (ctypes.c_void_p * len(v))(*v)
    ws = sgl.lora_linear_mx_workspace_bytes(32, 4, 72, 104, [64, 32], 16, True)
    assert ws >= sgl.lora_linear_mx_workspace_bytes(32, 4, 72, 104, [64, 32], 16, False) > 0
    ok = dict(x=0x10000, ldx=72, n=32, h=72, codes=0x20000, ldc=48, scales=0x30000, lds=4, out=104, wb=None,
              a=P(0x40000, 0x50000), b=P(0x60000, 0x70000), w=(ctypes.c_int * 2)(64, 32), s=2, r=16, buf=0x80000,
              y=0x90000, ldy=104, off=8, meta=None, ws=0xA0000, wsb=ws)

    def forward(**kw):
        a = dict(ok, **kw)
        m = a["meta"] or _fake_meta(sgl, 32)
        return L.lora_linear_mx(a["x"], a["ldx"], a["n"], a["h"], a["codes"], a["ldc"], a["scales"], a["lds"], a["out"],
                                a["wb"], a["a"], a["b"], None, a["w"], a["s"], a["r"], a["buf"], a["y"], a["ldy"],
                                a["off"], ctypes.byref(m), 1.0, 1, a["ws"], a["wsb"], None)

    def backward(**kw):
        a = dict(ok, **kw)
        m = a["meta"] or _fake_meta(sgl, 32)
        return L.lora_linear_mx_backward(a["y"], a["ldy"], a["x"], a["ldx"], a["n"], a["h"], a["codes"], a["ldc"],
                                         a["scales"], a["lds"], a["out"], a["a"], a["b"], a["w"], a["s"], a["r"],
                                         a["buf"], 0xB0000, 0xC0000, 72, P(0xD0000, 0xE0000), P(0xF0000, 0x100000), None,
                                         a["off"], ctypes.byref(m), 1.0, a["ws"], a["wsb"], None)
    for call in (forward, backward):
        assert call(ldc=32) == sgl.LORA_ERR_SHAPE and call(ldc=56) == sgl.LORA_ERR_SHAPE
        assert call(lds=2) == sgl.LORA_ERR_SHAPE and call(lds=6) == sgl.LORA_ERR_SHAPE
        assert call(h=76) == sgl.LORA_ERR_SHAPE and call(out=100) == sgl.LORA_ERR_SHAPE and call(off=16) == sgl.LORA_ERR_SHAPE
        assert call(n=31) == sgl.LORA_ERR_NUM_TOKENS and call(r=12) == sgl.LORA_ERR_SHAPE and call(s=9) == sgl.LORA_ERR_SLICES
        assert call(codes=None) == sgl.LORA_ERR_NULL and call(scales=None) == sgl.LORA_ERR_NULL
        assert call(codes=0x20008) == sgl.LORA_ERR_ALIGN and call(scales=0x30002) == sgl.LORA_ERR_ALIGN
        assert call(ldc=(1 << 25) + 16) == sgl.LORA_ERR_SHAPE
        assert call(ws=0xA0010) == sgl.LORA_ERR_BUFFER and call(wsb=256) == sgl.LORA_ERR_BUFFER
        assert call(x=0x10008) == sgl.LORA_ERR_ALIGN and call(y=None) == sgl.LORA_ERR_NULL
    assert forward(n=0, meta=_fake_meta(sgl, 0)) == sgl.LORA_OK
    assert sgl.lib.lora_linear_mx_workspace_bytes(32, 4, 72, 100, ok["w"], 2, 16, 1) == 0
    with pytest.raises(sgl.LoraError):
        sgl.lora_mx_row_bytes(12)


@pytest.mark.gpu
def test_refusals_of_the_binding():
    sgl = lib()
    c = MxCase(n=10, hidden=72, widths=[72], rank=8, loras=3)
    r = MxRun(c)
    for name, bad in (("codes", r.codes.cpu()), ("codes", r.codes.to(torch.int32)), ("scales", r.scales.float())):
        keep = getattr(r, name)
        setattr(r, name, bad)
        for call in (r.forward, r.backward):
            with pytest.raises(TypeError):
                call()
        setattr(r, name, keep)
    for name, bad in (("codes", r.codes[:, :32]), ("codes", r.codes[:-8]), ("scales", r.scales[:-1])):
        keep = getattr(r, name)
        setattr(r, name, bad)
        for call in (r.forward, r.backward):
            with pytest.raises(sgl.LoraError):
                call()
        setattr(r, name, keep)
    with pytest.raises(TypeError):
        sgl.lora_mx_quantize(r.x.half(), r.codes[:10], r.scales[:10])
    with pytest.raises(sgl.LoraError):
        sgl.lora_mx_quantize(r.x, r.codes[:9], r.scales[:10])
