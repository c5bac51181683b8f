"""Calls at the same time: two batches on two streams, each with its metadata and
workspace, from one thread and from two, give what each gives alone.
"""
import os
import sys
import threading

import pytest
import torch

sys.path.insert(0, os.path.dirname(__file__))
import test_mx  # noqa: E402
from test_clip import tensors  # noqa: E402
from test_linear import lib  # noqa: E402


class Job:
    """Forward, backward and clipping of one batch."""

    def __init__(self, acts, n, seed):
        sgl = lib()
        # (K is too short for a shrink that adds its parts in no order)
        self.c = test_mx.MxCase(acts=acts, n=n, hidden=136, widths=[520, 72], rank=24, loras=6, seed=seed)
        self.r = test_mx.MxRun(self.c)
        self.grads = self.r.da + self.r.db + self.r.dbias
        self.out = [torch.empty_like(t) for t in self.grads]
        self.held = sgl.LoraGradients(self.grads, self.out)
        self.norms = torch.empty(6, device="cuda")
        self.ws = torch.empty(sgl.lora_clip_gradients_workspace_bytes(self.held, 6), dtype=torch.uint8, device="cuda")

    def run(self, stream=None):
        self.r.forward(stream=stream)
        self.r.backward(stream=stream)
        lib().lora_clip_gradients(self.held, self.norms, 1e-2, self.ws, stream=stream)

    def outputs(self):
        return [self.r.y, self.r.dx, self.norms] + self.grads + self.out

    def poison(self):
        for t in self.outputs():
            t.fill_(float("nan"))


@pytest.mark.gpu
@pytest.mark.parametrize("threads", [False, True])
@pytest.mark.parametrize("sizes", [(("bf16", 20), ("mxfp4", 20)), (("bf16", 90), ("mxfp4", 300)), (("bf16", 2000), ("mxfp4", 2000))])
def test_two_streams(sizes, threads):
    jobs = [Job(acts, n, seed) for seed, (acts, n) in enumerate(sizes)]
    alone = []
    for j in jobs:
        j.run()
        test_mx.check(j.c, j.r.outputs())
        alone.append([t.clone() for t in j.outputs()])
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(3):
        for j in jobs:
            j.poison()
        torch.cuda.synchronize()

        def go(j, s):
            for _ in range(5):
                j.run(s)
        if threads:
            ts = [threading.Thread(target=go, args=p) for p in zip(jobs, streams)]
            for t in ts:
                t.start()
            for t in ts:
                t.join()
        else:
            for _ in range(5):
                for j, s in zip(jobs, streams):
                    j.run(s)
        torch.cuda.synchronize()
        for j, want in zip(jobs, alone):
            assert all(torch.equal(a, b) for a, b in zip(j.outputs(), want))


@pytest.mark.gpu
def test_many_lists_at_once():
    """Clipping of lists that need several launches, in place, on four streams."""
    sgl = lib()
    sets = [tensors([(4, 40 + i) for i in range(300)], (torch.float32, torch.bfloat16), 4, seed=k) for k in range(4)]
    want = []
    for t in sets:
        dev = [v.cuda() for v in t]
        norms = torch.empty(4, device="cuda")
        ws = torch.empty(sgl.lora_clip_gradients_workspace_bytes(dev, 4), dtype=torch.uint8, device="cuda")
        sgl.lora_clip_gradients(dev, norms, 1.0, ws)
        torch.cuda.synchronize()
        want.append([norms] + dev)
    jobs = []
    for t in sets:
        dev = [v.cuda() for v in t]
        held = sgl.LoraGradients(dev)
        jobs.append((held, torch.empty(4, device="cuda"),
                     torch.empty(sgl.lora_clip_gradients_workspace_bytes(held, 4), dtype=torch.uint8, device="cuda"), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for held, norms, ws, s in jobs:
        sgl.lora_clip_gradients(held, norms, 1.0, ws, stream=s)
    torch.cuda.synchronize()
    for (held, norms, _, _), w in zip(jobs, want):
        assert all(torch.equal(a, b) for a, b in zip([norms] + held.grads, w))
