"""Gradients and results anywhere in one buffer, in any order, some in place, some empty,
some read twice: what overlaps is refused and nothing is written, and everything else
gives the formula's results and leaves the rest of the buffer as it was.

Tolerances are those of test_clip.py.
"""
import os
import random
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(__file__))
from test_clip import compare  # noqa: E402
from test_linear import lib  # noqa: E402

WORDS = 400         # of the buffer, 4 bytes each


def spans(rng):
    """(gradient's, result's) first word, words and type of a few tensors."""
    out = []
    for _ in range(rng.randint(1, 5)):
        size, at = rng.choice((0, 1, 3, 8, 17, 40)), rng.randrange(WORDS - 40)
        out.append((at, at if rng.random() < 0.3 else rng.randrange(WORDS - 40), size,
                    rng.choice((torch.bfloat16, torch.float32))))
    return out


def overlap(a, b, n, m):
    return n > 0 and m > 0 and a < b + m and b < a + n


def refused(t):
    return any((i != j and overlap(p[1], q[1], p[2], q[2])) or (q[0] != q[1] and overlap(p[1], q[0], p[2], q[2]))
               for i, p in enumerate(t) for j, q in enumerate(t))


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(4))
def test_any_layout(seed):
    sgl = lib()
    rng = random.Random(seed)
    seen = {True: 0, False: 0}
    flat = torch.empty(WORDS, device="cuda")
    while min(seen.values()) < 40:
        t = spans(rng)
        bad = refused(t)
        if seen[bad] >= 40:
            continue
        seen[bad] += 1
        # ordinary numbers as either type
        flat.view(torch.bfloat16).copy_(torch.randn(2 * WORDS, generator=torch.Generator().manual_seed(len(t) + seed)))
        part = lambda at, size, kind: flat[at:at + size].view(kind)
        grads, out = [part(p[0], p[2], p[3]) for p in t], [part(p[1], p[2], p[3]) for p in t]
        given, before = [g.cpu().clone() for g in grads], flat.cpu().clone()
        norms = torch.empty(1, device="cuda")
        ws = torch.empty(sgl.lora_clip_gradients_workspace_bytes(grads), dtype=torch.uint8, device="cuda")
        if bad:
            with pytest.raises(sgl.LoraError) as e:
                sgl.lora_clip_gradients(grads, norms, 1.0, ws, out=out)
            assert e.value.status == sgl.LORA_ERR_BUFFER
            kept = torch.ones(WORDS, dtype=torch.bool)
        else:
            sgl.lora_clip_gradients(grads, norms, 1.0, ws, out=out)
            compare(given, norms, out, 1, 1.0)
            kept = torch.ones(WORDS, dtype=torch.bool)
            for p in t:
                kept[p[1]:p[1] + p[2]] = False
        assert torch.equal(flat.cpu().view(torch.int32)[kept], before.view(torch.int32)[kept])
