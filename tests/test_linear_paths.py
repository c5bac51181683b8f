"""lora_linear and its backward pass at the sizes where another kernel, tile or
walk is chosen, against the formulas in 64 bits; inputs, references and
tolerances as in test_linear."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(__file__))
from test_linear import Case, Run, check, lib  # noqa: E402

ALL = ("y", "dx", "s", "u", "da", "db", "dbias")


def _counts(n, counts):
    """ids of n tokens in a scattered order: counts[id] of each, the rest none."""
    ids = torch.full((n,), -1, dtype=torch.int64)
    at = 0
    for m, c in counts.items():
        ids[at:at + c] = m
        at += c
    return ids[torch.randperm(n, generator=torch.Generator().manual_seed(n))]


FEW = {   # up to 32 tokens: the two launches without a sort
    "15": dict(n=15, hidden=72, widths=[40, 16], rank=8, loras=3),
    "16": dict(n=16, hidden=1032, widths=[264, 8], rank=128, loras=5, offset=8, extra=16),
    "17": dict(n=17, hidden=520, widths=[136], rank=72, loras=4, stride=16),
    "31, no bias": dict(n=31, hidden=2056, widths=[8, 8, 8], rank=16, loras=40, bias=False),
    "32, one adapter": dict(n=32, hidden=8, widths=[72], rank=24, loras=1, none=0.0),
    "20, none": dict(n=20, hidden=136, widths=[72], rank=16, loras=4, none=1.0),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(FEW))
def test_few_tokens(name):
    c = Case(**FEW[name])
    r = Run(c)
    r.forward()
    r.backward()
    first = r.outputs()
    check(c, first)
    r.forward()
    again = r.outputs()
    assert torch.equal(first["y"], again["y"])      # no atomics on this path


TILES = {   # (case, results that the tile in question makes)
    "64 x 128, y": (dict(n=129, hidden=72, widths=[12800, 8], rank=40, loras=7), ("y", "s")),
    "64 x 128, dx": (dict(n=129, hidden=12808, widths=[40, 24], rank=16, loras=7), ("dx", "u")),
    "128 x 128, y": (dict(n=520, hidden=136, widths=[8000, 200], rank=16, loras=5), ("y", "s")),
    "128 x 128, dx": (dict(n=520, hidden=8200, widths=[72, 64], rank=72, loras=5), ("dx", "u")),
    "256 x 256, ranks up to 16": (dict(n=2050, hidden=200, widths=[5200, 72], rank=8, loras=90), ("y", "s")),
    "256 x 256, dx, many slices": (dict(n=2050, hidden=5272, widths=[8, 16, 24, 72], rank=128, loras=30), ("dx", "u")),
    "s packed by the sorted tokens": (dict(n=200, hidden=136, widths=[72, 40], rank=40, loras=6), ALL),
    "s by the shrink kernels": (dict(n=800, hidden=136, widths=[72, 40], rank=40, loras=6), ALL),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(TILES))
def test_tiles(name):
    kw, keys = TILES[name]
    c = Case(**kw)
    r = Run(c)
    r.forward()
    r.backward()
    check(c, r.outputs(), keys)


# gradients of adapters with 1, 63, 64, 65, 127, 128, 129 and 300 tokens: the walk
# with the packed rows kept in LDS, one and two K steps of it, and the other one
COUNTS = {0: 1, 2: 63, 3: 64, 5: 65, 6: 127, 7: 128, 9: 129, 10: 300}


@pytest.mark.gpu
@pytest.mark.parametrize("rank", [8, 32, 64, 128])
def test_lengths_of_segments(rank):
    n = sum(COUNTS.values()) + 23
    c = Case(n=n, hidden=200, widths=[136, 8], rank=rank, loras=12, ids=_counts(n, COUNTS))
    r = Run(c)
    r.forward()
    r.backward()
    check(c, r.outputs())


@pytest.mark.gpu
@pytest.mark.parametrize("rank,hidden,loras", [(8, 1032, 1023), (72, 520, 600)])
def test_runs_of_tiles(rank, hidden, loras):
    """So many adapters that a workgroup takes several tiles of one."""
    counts = {1: 40, loras - 1: 70, loras // 2: 1, 7: 150}
    c = Case(n=270, hidden=hidden, widths=[264], rank=rank, loras=loras, ids=_counts(270, counts))
    r = Run(c)
    r.forward()
    r.backward()
    check(c, r.outputs(), ("da", "db", "dbias"))


@pytest.mark.gpu
@pytest.mark.parametrize("n,rank", [(20, 16), (20, 40), (200, 40), (200, 8)])
def test_not_finite_stays_where_it_belongs(n, rank):
    c = Case(n=n, hidden=136, widths=[136, 40], rank=rank, loras=5)
    c.ids[:5] = torch.arange(5, dtype=torch.int32)
    r = Run(c)
    r.forward()
    r.backward()
    clean = r.outputs()
    bad = 3
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
def test_graph_replays_of_one_token():
    c = Case(n=1, hidden=1032, widths=[136, 72], rank=16, loras=6, none=0.0)
    r = Run(c)
    r.forward()
    eager = r.outputs()["y"]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r.forward()
    for _ in range(4):
        r.y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(r.outputs()["y"], eager)
        r.x.mul_(1.0)   # eager work between the replays


def test_widths_past_the_limit_are_refused():
    sgl = lib()
    assert sgl.lora_linear_workspace_bytes(16, 4, 1 << 24, [64], 8) > 0
    with pytest.raises(sgl.LoraError):
        sgl.lora_linear_workspace_bytes(16, 4, (1 << 24) + 8, [64], 8)


@pytest.mark.gpu
@pytest.mark.parametrize("n,loras,widths,rank", [(38, 26, [24, 48, 56], 80), (70, 40, [72, 8], 8), (130, 90, [136], 128),
                                                 (64, 4, [40], 16), (64, 3, [40], 16)])
def test_many_adapters_in_a_tile(n, loras, widths, rank):
    """Tiles that meet more and fewer adapters than a step of the walk is worth, y and dx."""
    c = Case(n=n, hidden=136, widths=widths, rank=rank, loras=loras, offset=8, extra=8)
    r = Run(c)
    r.forward()
    r.backward()
    check(c, r.outputs())
    r.a[0][0] = float("nan")        # what is not finite stays with its adapter's tokens
    r.b[0][0] = float("inf")
    before = r.outputs()
    r.forward()
    r.backward()
    after = r.outputs()
    rows = c.ids != 0
    assert torch.equal(before["y"][rows], after["y"][rows]) and torch.equal(before["dx"][rows], after["dx"][rows])
