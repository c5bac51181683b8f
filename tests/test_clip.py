"""lora_clip_gradients against the formulas in 64 bits on the CPU.

Tolerances: a square and a sum in double are off by 2^-53 each, which is nothing
beside the norm's rounding to float32, 2^-24 of it.  The factor is computed from
the norm in double and rounded to float32 (2^-24), the product is rounded to
float32 (2^-24) and, for bfloat16, once more (2^-8): in all 2^-8 + 2^-23 or 2^-23 of the
value, times 1 + 2^-6 for the products of these; a result that is subnormal in its
type is off by half of that type's quantum beside (2^-134, 2^-150).
"""
import ctypes
import math
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(__file__))
from test_linear import lib  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


def reference(grads, groups, limit):
    total = torch.zeros(groups, dtype=torch.float64)
    for t in grads:
        total += t.double().reshape(groups, -1).square().sum(1)
    norms = total.sqrt()
    factor = torch.where(torch.isfinite(norms), torch.clamp(limit / (norms + 1e-6), max=1.0), torch.ones_like(norms))
    return norms, factor, [(t.double().reshape(groups, -1) * factor[:, None]).reshape(t.shape) for t in grads]


def compare(grads, norms, out, groups, limit):
    want, factor, scaled = reference(grads, groups, limit)
    beyond = want >= 2.0 ** 128 * (1 - 2.0 ** -25)            # of float32: infinite there
    assert torch.isinf(norms.cpu()[beyond]).all()
    assert torch.allclose(norms.cpu().double()[~beyond], want[~beyond], rtol=2.0 ** -24 * (1 + 2.0 ** -6), atol=2.0 ** -150)
    for i, (t, o, v) in enumerate(zip(grads, out, scaled)):
        o = o.cpu()
        rel, quantum = (2.0 ** -8 + 2.0 ** -23, 2.0 ** -134 + 2.0 ** -150) if t.dtype is BF16 else (2.0 ** -23, 2.0 ** -150)
        off = ((o.double() - v).abs() / (v.abs() * rel * (1 + 2.0 ** -6) + quantum)).nan_to_num(nan=0.0)
        assert torch.equal(torch.isfinite(o), torch.isfinite(v)), i
        assert off.numel() == 0 or off.max().item() <= 1, (i, off.max().item())
        kept = (factor == 1)
        assert torch.equal(o.reshape(groups, -1)[kept], t.reshape(groups, -1)[kept]), i


def run(grads, groups, limit, in_place=False, out=None, workspace=None, **kw):
    sgl = lib()
    dev = [t.cuda() for t in grads]
    if out is None:
        out = dev if in_place else [torch.full_like(t, float("nan")) for t in dev]
    norms = torch.full((groups,), float("nan"), dtype=F32, device="cuda")
    if workspace is None:
        workspace = torch.full((sgl.lora_clip_gradients_workspace_bytes(dev, groups),), 0xFF, dtype=torch.uint8, device="cuda")
    sgl.lora_clip_gradients(dev, norms, limit, workspace, out=None if in_place else out, **kw)
    torch.cuda.synchronize()
    return norms, out, dev


def tensors(shapes, dtypes, groups=1, seed=0, spread=0.0):
    g = torch.Generator().manual_seed(seed)
    size = torch.exp2(spread * torch.randn(groups, generator=g, dtype=torch.float64))
    out = []
    for i, s in enumerate(shapes):
        t = torch.randn(s, generator=g, dtype=torch.float64)
        if groups > 1:
            t = (t.reshape(groups, -1) * size[:, None]).reshape(s)
        out.append(t.to(dtypes[i % len(dtypes)]))
    return out


SETS = {
    "one number": ([(1,)], 1),
    "odd sizes": ([(3,), (17, 5), (1, 1, 1), (1023,), (8191,), (33, 77)], 1),
    "an empty one among them": ([(5,), (0,), (0, 3), (9,)], 1),
    "a step of five adapters": ([(5, 8, 520), (5, 136, 8), (5, 136), (5, 8, 520), (5, 72, 8), (5, 72)], 5),
    "odd parts": ([(7, 3, 5), (7, 1), (7, 1001), (7, 4099)], 7),
    "many adapters": ([(1023, 9), (1023, 1)], 1023),
    "many tensors": ([(4, 40 + i) for i in range(300)], 4),
    "a long one": ([(300000, 41)], 1),
    "more sums than a workgroup adds": ([(5000001,)] * 20, 1),
    "several pieces a part": ([(3, 200003), (3, 99991)], 3),
}


@pytest.mark.gpu
@pytest.mark.parametrize("dtypes", [(BF16,), (F32,), (F32, BF16)], ids=["bf16", "fp32", "both"])
@pytest.mark.parametrize("name", list(SETS))
def test_against_formulas(name, dtypes):
    shapes, groups = SETS[name]
    grads = tensors(shapes, dtypes, groups, spread=2.0)
    norms, _, _ = reference(grads, groups, 1.0)
    for limit in (float(norms.median()), float(norms.max()) * 2, float(norms.min()) / 3, math.inf):
        for in_place in (False, True):
            got, out, dev = run(grads, groups, limit, in_place)
            compare(grads, got, out, groups, limit)
            if not in_place:
                assert all(torch.equal(d.cpu(), t) for d, t in zip(dev, grads))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_starts_that_are_not_aligned(dtype):
    """Parts of one buffer at any element, results at other ones."""
    sgl = lib()
    g = torch.Generator().manual_seed(2)
    flat = torch.randn(70000, generator=g).to(dtype)
    dev, to = flat.cuda(), torch.full((70013,), 9.0, dtype=dtype, device="cuda")
    spans = [(1, 4), (7, 5000), (5001, 5002), (5003, 60000), (60001, 69998)]
    for shift in (0, 1, 3, 8, 13):
        to.fill_(9.0)
        grads, out = [dev[a:b] for a, b in spans], [to[a + shift:b + shift] for a, b in spans]
        norms = torch.empty(1, device="cuda")
        ws = torch.empty(sgl.lora_clip_gradients_workspace_bytes(grads), dtype=torch.uint8, device="cuda")
        sgl.lora_clip_gradients(grads, norms, 3.0, ws, out=out)
        compare([t.cpu() for t in grads], norms, out, 1, 3.0)
        rest = torch.ones(70013, dtype=torch.bool)
        for a, b in spans:
            rest[a + shift:b + shift] = False
        assert (to.cpu()[rest] == 9.0).all()


@pytest.mark.gpu
def test_extreme_magnitudes():
    """Squares beyond float32 on both sides, subnormal numbers, zeros."""
    for dtype in (BF16, F32):
        for power in (127, 100, 64, 0, -63, -75, -100, -126, -133):
            t = [torch.ones(1000, dtype=torch.float64).mul_(2.0 ** power).to(dtype), torch.zeros(7, dtype=dtype)]
            for limit in (1e-3, 1.0, 3.0e38):
                got, out, _ = run(t, 1, limit)
                compare(t, got, out, 1, limit)
    zeros = [torch.zeros(100, dtype=F32), torch.zeros(9, dtype=BF16)]
    got, out, _ = run(zeros, 1, 1.0)
    assert (got == 0).all() and all((t == 0).all() for t in out)


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_not_finite_stays_in_its_group(bad):
    grads = tensors([(6, 5000), (6, 77)], (BF16, F32), 6)
    grads[1][2, 5] = bad
    for in_place in (False, True):
        got, out, _ = run(grads, 6, 1.0, in_place)
        assert not torch.isfinite(got[2]) and torch.isfinite(got[[0, 1, 3, 4, 5]]).all()
        for o, t in zip(out, grads):
            assert torch.equal(torch.nan_to_num(o[2].cpu()), torch.nan_to_num(t[2]))
        keep = [0, 1, 3, 4, 5]
        compare([t[keep] for t in grads], got[keep], [o[keep] for o in out], 5, 1.0)


@pytest.mark.gpu
def test_no_tensors():
    sgl = lib()
    norms = torch.full((3,), 5.0, device="cuda")
    ws = torch.empty(sgl.lora_clip_gradients_workspace_bytes([], 3), dtype=torch.uint8, device="cuda")
    sgl.lora_clip_gradients([], norms, 1.0, ws)
    assert (norms.cpu() == 0).all()


@pytest.mark.gpu
def test_same_bits_again_and_replayed():
    """Two calls give the same bits; so does a captured one, replayed over other
    gradients on another stream with eager work between."""
    sgl = lib()
    shapes = [(4, 70001), (4, 8, 520), (4, 3)]
    first, second = tensors(shapes, (BF16, F32), 4, seed=1), tensors(shapes, (BF16, F32), 4, seed=2)
    dev = [t.cuda() for t in first]
    out = [torch.empty_like(t) for t in dev]
    held = sgl.LoraGradients(dev, out)
    norms = torch.empty(4, device="cuda")
    ws = torch.full((sgl.lora_clip_gradients_workspace_bytes(held, 4),), 0xFF, dtype=torch.uint8, device="cuda")
    eager = []
    for grads in (first, second):
        for t, v in zip(dev, grads):
            t.copy_(v)
        both = []
        for _ in range(2):
            ws.fill_(0xFF)
            sgl.lora_clip_gradients(held, norms, 1.0, ws)
            both.append([norms.clone()] + [t.clone() for t in out])
        assert all(torch.equal(a, b) for a, b in zip(*both))
        compare(grads, norms, out, 4, 1.0)
        eager.append(both[0])
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        sgl.lora_clip_gradients(held, norms, 1.0, ws)
    for k in range(4):
        for t, v in zip(dev, (first, second)[k % 2]):
            t.copy_(v)
        ws.fill_(0x11 * k)
        for t in out:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager[k % 2], [norms] + out))


@pytest.mark.gpu
def test_tensors_that_moved_are_seen():
    sgl = lib()
    t = torch.full((100,), 2.0, device="cuda")
    held = sgl.LoraGradients([t])
    norms = torch.empty(1, device="cuda")
    ws = torch.empty(sgl.lora_clip_gradients_workspace_bytes(held), dtype=torch.uint8, device="cuda")
    t.data = torch.full((50,), 3.0, device="cuda")
    sgl.lora_clip_gradients(held, norms, 1.0, ws)
    assert abs(float(norms) - 3 * math.sqrt(50)) < 1e-4
    assert abs(float(t.norm()) - 1.0) < 1e-5


def test_refusals():
    sgl = lib()
    L = sgl.lib
    P = lambda *v: (ctypes.c_void_p * len(v))(*v)
    S = lambda *v: (ctypes.c_int64 * len(v))(*v)
    T = lambda *v: (ctypes.c_int * len(v))(*v)
    ok = dict(g=P(0x10000, 0x20000), o=P(0x30000, 0x40000), s=S(64, 32), t=T(0, 1), n=2, groups=4, limit=1.0, norms=0x50000,
              ws=0x60000, wsb=1 << 20)

    def call(**kw):
        a = dict(ok, **kw)
        return L.lora_clip_gradients(a["g"], a["o"], a["s"], a["t"], a["n"], a["groups"], a["limit"], a["norms"], a["ws"],
                                     a["wsb"], None)
    assert call(groups=0) == sgl.LORA_ERR_MAX_LORAS and call(groups=1024) == sgl.LORA_ERR_MAX_LORAS
    assert call(n=-1) == sgl.LORA_ERR_SLICES and call(n=65537) == sgl.LORA_ERR_SLICES
    assert call(groups=3) == sgl.LORA_ERR_SHAPE and call(s=S(64, -4)) == sgl.LORA_ERR_SHAPE
    assert call(t=T(0, 2)) == sgl.LORA_ERR_SHAPE
    for limit in (0.0, -1.0, math.nan):
        assert call(limit=limit) == sgl.LORA_ERR_SHAPE
    assert call(norms=None) == sgl.LORA_ERR_NULL and call(ws=None) == sgl.LORA_ERR_NULL
    assert call(g=P(0x10000, None)) == sgl.LORA_ERR_NULL and call(o=P(None, 0x40000)) == sgl.LORA_ERR_NULL
    assert call(g=None) == sgl.LORA_ERR_NULL and call(s=None) == sgl.LORA_ERR_NULL
    assert call(g=P(0x10001, 0x20000)) == sgl.LORA_ERR_ALIGN and call(o=P(0x30000, 0x40002)) == sgl.LORA_ERR_ALIGN
    assert call(norms=0x50002) == sgl.LORA_ERR_ALIGN
    assert call(ws=0x60080) == sgl.LORA_ERR_BUFFER and call(wsb=16) == sgl.LORA_ERR_BUFFER
    assert call(o=P(0x30000, 0x30000)) == sgl.LORA_ERR_BUFFER         # the same place twice
    assert call(o=P(0x30000, 0x3007c)) == sgl.LORA_ERR_BUFFER         # 64 bfloat16 end at 0x30080
    assert sgl.lib.lora_clip_gradients_workspace_bytes(ok["s"], ok["t"], 2, 3) == 0
    assert sgl.lib.lora_clip_gradients_workspace_bytes(ok["s"], ok["t"], 2, 4) > 0


def test_results_on_other_gradients_are_refused():
    sgl = lib()
    P = lambda *v: (ctypes.c_void_p * len(v))(*v)

    def call(g, o, sizes=(64, 32, 0), types=(0, 1, 1)):       # 0x80 bytes either, and nothing
        return sgl.lib.lora_clip_gradients(P(*g), P(*o), (ctypes.c_int64 * 3)(*sizes), (ctypes.c_int * 3)(*types), 3, 4, 1.0,
                                           0x50000, 0x60000, 1 << 20, None)
    a, b, c, d = 0x10000, 0x20000, 0x30000, 0x40000
    assert call((a, b, 0), (b, a, 0)) == sgl.LORA_ERR_BUFFER             # each on the other
    assert call((a, b, 0), (b, d, 0)) == sgl.LORA_ERR_BUFFER
    assert call((a, b, 0), (c, a, 0)) == sgl.LORA_ERR_BUFFER
    assert call((b, a, 0), (a, c, 0)) == sgl.LORA_ERR_BUFFER             # gradients out of order
    assert call((a, b, 0), (a + 16, c, 0)) == sgl.LORA_ERR_BUFFER        # a part of its own
    assert call((a + 16, b, 0), (a, c, 0)) == sgl.LORA_ERR_BUFFER
    assert call((a, b, 0), (c, b + 0x7c, 0)) == sgl.LORA_ERR_BUFFER      # its last number
    assert call((a, b, 0), (c, b - 0x7c, 0)) == sgl.LORA_ERR_BUFFER
    assert call((a, a, 0), (a, c, 0)) == sgl.LORA_ERR_BUFFER             # in place, and read elsewhere
    assert call((a, a + 0x40, 0), (c, a + 0x60, 0)) == sgl.LORA_ERR_BUFFER   # gradients that overlap


@pytest.mark.gpu
def test_results_between_the_gradients():
    # gradients and results side by side in one buffer, in no order, one in place, one read twice
    sgl = lib()
    flat = torch.arange(1, 97, dtype=torch.float32, device="cuda")
    at = lambda i: flat[8 * i:8 * i + 8]
    grads, out = [at(5), at(1), at(8), at(3), at(3)], [at(4), at(2), at(8), at(0), at(9)]
    want_in = [t.double() for t in grads]
    norm = torch.cat(want_in).norm()
    before = flat.clone()
    norms, ws = torch.empty(1, device="cuda"), torch.empty(sgl.lora_clip_gradients_workspace_bytes(grads), dtype=torch.uint8, device="cuda")
    sgl.lora_clip_gradients(grads, norms, 2.0, ws, out=out)
    assert abs(float(norms) - float(norm)) <= 2 ** -23 * float(norm)
    for w, o in zip(want_in, out):
        # the factor's rounding, the product's
        torch.testing.assert_close(o.double(), w * (2.0 / (norm + 1e-6)), rtol=3 * 2 ** -24, atol=0)
    kept = torch.ones(12, dtype=torch.bool)
    kept[[4, 2, 8, 0, 9]] = False
    assert torch.equal(flat.reshape(12, 8)[kept.cuda()], before.reshape(12, 8)[kept.cuda()])


@pytest.mark.gpu
def test_refusals_of_the_binding():
    sgl = lib()
    t = torch.ones((4, 6), device="cuda")
    norms, ws = torch.empty(4, device="cuda"), torch.empty(4096, dtype=torch.uint8, device="cuda")
    for bad in ([t.cpu()], [t.half()], [t, t.cpu()]):
        with pytest.raises(TypeError):
            sgl.lora_clip_gradients(bad, norms, 1.0, ws)
    for bad in ([t[:, ::2]], [t, t], [t[:3]], [t, t[1:]]):
        with pytest.raises(sgl.LoraError):
            sgl.lora_clip_gradients(bad, norms, 1.0, ws)
    with pytest.raises(TypeError):
        sgl.lora_clip_gradients([t], norms.double(), 1.0, ws)
    with pytest.raises(TypeError):
        sgl.lora_clip_gradients([t], norms, 1.0, ws, out=[t.to(BF16)])
    with pytest.raises(sgl.LoraError):
        sgl.lora_clip_gradients([t], norms, 1.0, ws, out=[t, t])
    assert (t == 1).all()
