"""A training step over a matrix in 4 bits, as it is used: quantize once, then
prepare, lora_linear_mx, lora_cross_entropy, both backward passes and
lora_clip_gradients, adapter by adapter, on one stream with one workspace for all of
them; eager, and captured and replayed.  Every call's outputs are checked against the
formulas in 64 bits on the inputs that it had, with the tolerances of its own tests.
"""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(__file__))
import test_clip  # noqa: E402
import test_linear  # noqa: E402
import test_mx  # noqa: E402
from test_linear import lib  # noqa: E402


class Step:
    def __init__(self, acts, n, hidden, widths, rank, loras, vocab, seed):
        sgl = lib()
        self.acts, self.loras = acts, loras
        self.case = c = test_mx.MxCase(acts=acts, n=n, hidden=hidden, widths=widths, rank=rank, loras=loras, seed=seed)
        dev = lambda ts: [None if t is None else t.cuda() for t in ts]
        g = torch.Generator().manual_seed(seed + 5)
        self.x, self.ids = c.x.cuda(), c.ids.cuda()
        self.a, self.b, self.bias, self.w_bias = dev(c.a), dev(c.b), dev(c.bias), c.w_bias.cuda()
        # the matrix as it is loaded, in bfloat16, and what the projection keeps of it
        w = (torch.randn((c.out, hidden), generator=g) * 0.05).to(torch.bfloat16)
        code_bytes, scale_bytes = sgl.lora_mx_row_bytes(hidden)
        self.codes = torch.empty((c.out, code_bytes), dtype=torch.uint8, device="cuda")
        self.scales = torch.empty((c.out, scale_bytes), dtype=torch.uint8, device="cuda")
        sgl.lora_mx_quantize(w.cuda(), self.codes, self.scales)
        c.w = test_mx.quantized(w.double())[2]
        self.head = (torch.randn((vocab, c.out), generator=g) * 0.05).to(torch.bfloat16).cuda()
        self.targets = torch.randint(-1, vocab, (n,), generator=g, dtype=torch.int32).cuda()
        S, bf16, f32 = len(widths), torch.bfloat16, torch.float32
        new = lambda shape, dt: torch.full(shape, float("nan"), dtype=dt, device="cuda")
        self.meta = sgl.LoraMeta(loras, n)
        self.buf, self.dbuf = new((S, n, rank), f32), new((S, n, rank), f32)
        self.y, self.dy, self.dx = new((n, c.out), bf16), new((n, c.out), bf16), new((n, hidden), bf16)
        self.loss, self.lse = new((n,), f32), new((n,), f32)
        self.dloss = torch.full((n,), 1.0 / n, device="cuda")
        self.da = [new(t.shape, bf16) for t in self.a]
        self.db = [new(t.shape, bf16) for t in self.b]
        self.dbias = [new(t.shape[:2], bf16) for t in self.b]
        self.grads = self.da + self.db + self.dbias
        self.out = [torch.full_like(t, float("nan")) for t in self.grads]
        self.held = sgl.LoraGradients(self.grads, self.out)
        self.norms = new((loras,), f32)
        size = max(sgl.lora_linear_mx_workspace_bytes(n, loras, hidden, c.out, widths, rank, True),
                   sgl.lora_cross_entropy_workspace_bytes(n, c.out, vocab, True),
                   sgl.lora_clip_gradients_workspace_bytes(self.held, loras))
        self.workspace = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
        self.limit = 1e-3

    def run(self):
        sgl, c, ws = lib(), self.case, self.workspace
        sgl.lora_prepare_meta(self.ids, self.meta)
        sgl.lora_linear_mx(self.x, self.codes, self.scales, self.w_bias, self.a, self.b, self.bias, self.buf, self.y,
                           self.meta, c.scale, ws, quantize_x=self.acts == "mxfp4")
        sgl.lora_cross_entropy(self.y, self.head, self.targets, self.loss, self.lse, ws)
        sgl.lora_cross_entropy_backward(self.y, self.head, self.targets, self.lse, self.dloss, self.dy, None, ws)
        sgl.lora_linear_mx_backward(self.dy, self.x, self.codes, self.scales, self.a, self.b, self.buf, self.dbuf,
                                    self.dx, self.da, self.db, self.dbias, self.meta, c.scale, ws)
        sgl.lora_clip_gradients(self.held, self.norms, self.limit, ws)

    def check(self):
        torch.cuda.synchronize()
        c = self.case
        c.dy = self.dy.cpu()
        host = lambda ts: [t.cpu().double() for t in ts]
        test_mx.check(c, {"y": self.y.cpu().double(), "dx": self.dx.cpu().double(), "da": host(self.da),
                          "db": host(self.db), "dbias": host(self.dbias)}, ("y", "dx", "da", "db", "dbias"))
        # the loss of the y that there is: float32 sums, off by 2^-22 (H + 8) of the logits' magnitudes at most
        y, head = self.y.cpu().double(), self.head.cpu().double()
        z, mag = y @ head.t(), (y.abs() @ head.abs().t()).amax(1)
        lse = torch.logsumexp(z, 1)
        assert ((self.lse.cpu().double() - lse).abs() <= 2.0 ** -22 * (c.out + 8) * (mag + lse.abs() + 1)).all()
        grads = [t.cpu() for t in self.grads]
        norms, factor, _ = test_clip.reference(grads, self.loras, self.limit)
        assert (factor < 1).any()
        test_clip.compare(grads, self.norms, self.out, self.loras, self.limit)


@pytest.mark.gpu
@pytest.mark.parametrize("acts,n", [("bf16", 20), ("bf16", 70), ("mxfp4", 20), ("mxfp4", 300)])
def test_step(acts, n):
    step = Step(acts, n, hidden=136, widths=[72, 64], rank=24, loras=5, vocab=203, seed=n)
    step.run()
    step.check()
    first = [t.clone() for t in step.out]
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step.run()
    for k in range(3):
        for t in step.out + step.grads + [step.y, step.dy, step.dx]:
            t.fill_(float("nan"))
        step.workspace.fill_(0x55 * k)
        (torch.ones(1000, device="cuda") * k).sum().item()       # eager work between the replays
        graph.replay()
        step.check()
    assert all(t.shape == o.shape for t, o in zip(first, step.out))
