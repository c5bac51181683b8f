"""Training steps of the adapters of a batch of requests: one projection that they
share, its adapters, and the vocabulary's cross entropy on top.

    python examples/adapter_step.py [steps]

A batch of 192 tokens belongs to five adapters and some to none.  Every step runs
lora_linear, lora_cross_entropy and their backward passes on one stream with
buffers made once, and moves the adapters (float32 copies, rounded to bfloat16)
against their gradients; the projection and the vocabulary matrix stay frozen.
Prints the mean loss of every step.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import segmented_gather_lora_amd as sgl  # noqa: E402


def train(steps=12, tokens=192, hidden=256, width=264, rank=16, loras=5, vocab=1003, rate=10.0, seed=0):
    """Mean losses of the steps' forward passes."""
    g = torch.Generator("cpu").manual_seed(seed)
    dev = dict(device="cuda")

    def normal(*shape, sigma=1.0):
        return (torch.randn(shape, generator=g) * sigma).to(torch.bfloat16).cuda()
    x, w, head = normal(tokens, hidden), normal(width, hidden, sigma=0.05), normal(vocab, width, sigma=0.05)
    # the adapters: A at random, B zero, kept in float32 between the steps
    a32 = (torch.randn((loras, rank, hidden), generator=g) * 0.05).cuda()
    b32 = torch.zeros((loras, width, rank), **dev)
    ids = torch.randint(-1, loras, (tokens,), generator=g, dtype=torch.int32).cuda()
    targets = torch.randint(0, vocab, (tokens,), generator=g, dtype=torch.int32)
    targets[::7] = -1                                   # prompts' positions do not count
    counted = int((targets >= 0).sum())
    targets = targets.cuda()
    scale = 1.0

    meta = sgl.LoraMeta(loras, tokens)
    buf = torch.empty((1, tokens, rank), dtype=torch.float32, **dev)
    dbuf = torch.empty_like(buf)
    y = torch.empty((tokens, width), dtype=torch.bfloat16, **dev)
    dy = torch.empty_like(y)
    loss, lse = torch.empty(tokens, **dev), torch.empty(tokens, **dev)
    dloss = torch.full((tokens,), 1.0 / counted, **dev)
    da, db = torch.empty_like(a32, dtype=torch.bfloat16), torch.empty_like(b32, dtype=torch.bfloat16)
    linear = torch.empty(sgl.lora_linear_workspace_bytes(tokens, loras, hidden, [width], rank, True),
                         dtype=torch.uint8, **dev)
    entropy = torch.empty(sgl.lora_cross_entropy_workspace_bytes(tokens, width, vocab, True), dtype=torch.uint8, **dev)

    sgl.lora_prepare_meta(ids, meta)
    losses = []
    for _ in range(steps):
        a, b = a32.to(torch.bfloat16), b32.to(torch.bfloat16)
        sgl.lora_linear(x, w, None, [a], [b], None, buf, y, meta, scale, linear)
        sgl.lora_cross_entropy(y, head, targets, loss, lse, entropy)
        sgl.lora_cross_entropy_backward(y, head, targets, lse, dloss, dy, None, entropy)
        sgl.lora_linear_backward(dy, x, w, [a], [b], buf, dbuf, None, [da], [db], None, meta, scale, linear)
        a32 -= rate * da.float()
        b32 -= rate * db.float()
        losses.append(float(loss.sum()) / counted)
    return losses


if __name__ == "__main__":
    for step, value in enumerate(train(int(sys.argv[1]) if len(sys.argv) > 1 else 12)):
        print("step %2d  loss %.4f" % (step, value))
