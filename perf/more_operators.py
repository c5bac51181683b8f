"""A projection held in microscaled 4-bit numbers, with the adapters of many
requests, and the norms of the adapters' gradients, as cases that can be timed.

``quantize``: rows of numbers to codes of 4 bits (E2M1) with a power of two
(E8M0) for every 32 of a row, and back to the numbers that they stand for.

``linear``: the projection that every request shares, held as such codes, with
the low-rank adapters of many requests added in the same product.  The
activations stay as they are (``acts: "bf16"``) or are quantized in the call as
the weights were (``acts: "mxfp4"``, serving).  ``pass: "train"`` is a training
step of the adapters over the frozen codes: forward, then the gradients of the
input, the adapters and their bias.

``clip``: the norm of all gradients of a training step, over many tensors, or
one norm for each adapter over its own matrices in all of them (every adapter is
a training of its own), and the gradients scaled down to a largest norm.

``run`` computes them from elementary torch operations in 32 bits, or, where
``own`` is set, with the library's calls.  ``exact`` computes them in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

DEVICE = "cuda"
SIGMA_W = 0.02          # weights ~N(0, 0.02), as in the repository's workloads
BLOCK = 32              # numbers that share a power of two
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)     # E2M1, code 0..7; 8 more is the sign
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- cases

def _quantize(name, rows, cols, kind):
    return {"name": name, "op": "quantize", "rows": rows, "cols": cols, "type": kind}


def _linear(name, step, acts, tokens, hidden, slices, rank, loras, ids, none, bias):
    return {"name": name, "op": "linear", "pass": step, "acts": acts, "tokens": tokens, "hidden": hidden,
            "slices": ",".join(str(w) for w in slices), "rank": rank, "loras": loras, "ids": ids, "none": none,
            "bias": bias}


def _clip(name, layers, hidden, slices, rank, loras, kind, per_lora, bias):
    return {"name": name, "op": "clip", "layers": layers, "hidden": hidden,
            "slices": ",".join(str(w) for w in slices), "rank": rank, "loras": loras, "type": kind,
            "per_lora": per_lora, "bias": bias}


def listed():
    return [
        # the activations of a small decode step: latency alone
        _quantize("quantize 16 rows", 16, 4096, "bf16"),
        # rows that end inside a block of 32, from float32
        _quantize("quantize odd", 1003, 1032, "fp32"),
        # a model's gate and up projections as they are loaded
        _quantize("quantize gate up", 28672, 4096, "bf16"),
        # one request's next token through a q/k/v projection
        _linear("linear one token", "forward", "bf16", 1, 4096, (4096, 1024, 1024), 16, 32, "uniform", 0.0, False),
        # a decode step of 256 requests over 32 adapters
        _linear("linear decode", "forward", "bf16", 256, 4096, (4096, 1024, 1024), 16, 32, "uniform", 0.10, False),
        # prompts of 512 tokens each, with biases, activations in 4 bits too
        _linear("linear prefill 4 bits", "forward", "mxfp4", 8192, 4096, (4096, 1024, 1024), 64, 8, "runs", 0.0, True),
        # nothing a multiple of a tile or of a block, a slice of 8 columns
        _linear("linear odd 4 bits", "forward", "mxfp4", 1003, 1032, (264, 8, 520), 24, 9, "uniform", 0.25, True),
        # gate and up projections, sequences of 256 tokens dealt to 16 adapters
        _linear("linear train gate up", "train", "bf16", 4096, 4096, (14336, 14336), 32, 16, "dealt", 0.0, False),
        # a small ragged step with biases
        _linear("linear train odd", "train", "bf16", 517, 520, (136, 72), 8, 5, "uniform", 0.20, True),
        # the gradients of that small step, five trainings side by side
        _clip("clip odd", 1, 520, (136, 72), 8, 5, "bf16", True, True),
        # one adapter's gradients over 32 layers of q/k/v, 192 tensors, one norm
        _clip("clip 32 layers", 32, 4096, (4096, 1024, 1024), 16, 1, "fp32", False, False),
        # the largest mixed step's gradients: 128 trainings of rank 128
        _clip("clip 128 adapters", 1, 8192, (8192, 1024, 1024), 128, 128, "bf16", True, False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    """One more case of the ranges: widths in steps of 8 (the library's rows are
    16-byte aligned), tokens 1..16384, any number of tensors up to a few hundred."""
    most = max(_cost(c) for c in listed())
    while True:
        kind = rng.random()
        if kind < 0.25:
            case = _quantize("", _log(rng, 1, 32768), 8 * _log(rng, 1, 2048), rng.choice(("bf16", "fp32")))
        elif kind < 0.75:
            step = rng.choice(("forward", "forward", "train"))
            slices = [8 * _log(rng, 1, 1024) for _ in range(rng.choice((1, 1, 2, 3)))]
            case = _linear("", step, rng.choice(("bf16", "mxfp4")) if step == "forward" else "bf16",
                           _log(rng, 1, 16384), 8 * _log(rng, 16, 1024), slices, 8 * rng.randint(1, 16),
                           _log(rng, 1, 128), rng.choice(("uniform", "runs", "dealt")), rng.choice((0.0, 0.1, 0.3)),
                           rng.random() < 0.4)
        else:
            slices = [8 * _log(rng, 1, 1024) for _ in range(rng.choice((1, 2, 3)))]
            case = _clip("", _log(rng, 1, 40), 8 * _log(rng, 16, 1024), slices, 8 * rng.randint(1, 16),
                         _log(rng, 1, 128), rng.choice(("bf16", "fp32")), rng.random() < 0.5, rng.random() < 0.4)
        del case["name"]
        if _cost(case) <= most and _bytes_held(case) < 12e9:
            return case


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def _bytes_held(case):
    """Bytes of the largest things that the plain form holds."""
    if case["op"] == "quantize":
        return 40.0 * case["rows"] * case["cols"]
    if case["op"] == "clip":
        return 16.0 * _grad_elements(case)
    out = sum(_widths(case))
    wide = out + case["hidden"]
    return (24.0 * out * case["hidden"] + 40.0 * case["tokens"] * wide
            + 8.0 * case["loras"] * case["rank"] * wide * len(_widths(case)))


# ---------------------------------------------------------------- inputs

def _widths(case):
    return [int(w) for w in case["slices"].split(",")]


def _normal(gen, shape, sigma=1.0, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device=DEVICE, dtype=torch.float32).mul_(sigma).to(dtype)


def _mapping(case, seed):
    """Adapter ids of the tokens (-1: none), on the host."""
    gen = torch.Generator("cpu").manual_seed(seed * 7919 + 13)
    n, loras = case["tokens"], case["loras"]
    if case["ids"] == "uniform":
        ids = torch.randint(0, loras, (n,), generator=gen)
    else:
        run = 512 if case["ids"] == "runs" else 256
        runs = (n + run - 1) // run
        if case["ids"] == "runs":
            of_run = torch.randint(0, loras, (runs,), generator=gen)
        else:
            of_run = torch.randperm(runs, generator=gen) % loras
        ids = of_run.repeat_interleave(run)[:n]
    none = int(round(case["none"] * n))
    if none:
        ids[torch.randperm(n, generator=gen)[:none]] = -1
    return ids.to(torch.int32)


def _prepare_quantize(case, seed):
    gen = torch.Generator(DEVICE).manual_seed(seed)
    rows, cols = case["rows"], case["cols"]
    # rows of different magnitudes, and one column in 64 that stands out, as activations have them
    x = torch.randn((rows, cols), generator=gen, device=DEVICE, dtype=torch.float32)
    x *= torch.exp2(4.0 * torch.randn((rows, 1), generator=gen, device=DEVICE))
    x *= torch.where(torch.rand(cols, generator=gen, device=DEVICE) < 1 / 64, 20.0, 1.0)
    st = {"case": case, "x": x.to(TYPES[case["type"]])}
    if own:
        import segmented_gather_lora_amd as sgl
        code_bytes, scale_bytes = sgl.lora_mx_row_bytes(cols)
        st["codes"] = torch.empty((rows, code_bytes), dtype=torch.uint8, device=DEVICE)
        st["scales"] = torch.empty((rows, scale_bytes), dtype=torch.uint8, device=DEVICE)
        st["out"] = torch.empty((rows, cols), dtype=torch.bfloat16, device=DEVICE)
    return st


def _prepare_linear(case, seed):
    gen = torch.Generator(DEVICE).manual_seed(seed)
    n, hidden, rank, loras, widths = case["tokens"], case["hidden"], case["rank"], case["loras"], _widths(case)
    out = sum(widths)
    ids = _mapping(case, seed)
    # the plan of a batch: every present adapter's tokens, padded to the longest with the index n
    present = torch.unique(ids[ids >= 0]).long()
    longest = max([int((ids == m).sum()) for m in present.tolist()], default=0)
    plan = torch.full((len(present), longest), n, dtype=torch.int64)
    for j, m in enumerate(present.tolist()):
        of = torch.nonzero(ids == m).flatten()
        plan[j, :len(of)] = of
    codes, scales = _to_blocks(_normal(gen, (out, hidden), SIGMA_W).float())
    st = {"case": case, "ids": ids.to(DEVICE), "present": present.to(DEVICE), "plan": plan.to(DEVICE),
          "scale": 2.0 / math.sqrt(rank), "widths": widths, "codes": codes, "scales": scales,
          "x": _normal(gen, (n, hidden)),
          "a": [_normal(gen, (loras, rank, hidden), SIGMA_W) for _ in widths],
          "b": [_normal(gen, (loras, w, rank), SIGMA_W) for w in widths],
          "w_bias": _normal(gen, (out,), 0.1) if case["bias"] else None,
          "bias": [_normal(gen, (loras, w), 0.1) for w in widths] if case["bias"] else None}
    if case["pass"] == "train":
        st["dy"] = _normal(gen, (n, out), 0.01)
    if own:
        import segmented_gather_lora_amd as sgl
        train = case["pass"] == "train"
        st["meta"] = sgl.LoraMeta(loras, n)
        sgl.lora_prepare_meta(st["ids"], st["meta"])
        st["buf"] = torch.empty((len(widths), n, rank), dtype=torch.float32, device=DEVICE)
        st["y"] = torch.empty((n, out), dtype=torch.bfloat16, device=DEVICE)
        st["workspace"] = torch.zeros(
            sgl.lora_linear_mx_workspace_bytes(n, loras, hidden, out, widths, rank, train),
            dtype=torch.uint8, device=DEVICE)
        if train:
            st["dbuf"] = torch.empty_like(st["buf"])
            st["dx"] = torch.empty_like(st["x"])
            st["da"] = [torch.empty_like(t) for t in st["a"]]
            st["db"] = [torch.empty_like(t) for t in st["b"]]
            st["dbias"] = None if st["bias"] is None else [torch.empty_like(t) for t in st["bias"]]
    return st


def _grad_shapes(case):
    loras, rank, hidden = case["loras"], case["rank"], case["hidden"]
    one = []
    for w in _widths(case):
        one += [(loras, rank, hidden), (loras, w, rank)] + ([(loras, w)] if case["bias"] else [])
    return one * case["layers"]


def _grad_elements(case):
    return sum(math.prod(s) for s in _grad_shapes(case))


def _prepare_clip(case, seed):
    gen = torch.Generator(DEVICE).manual_seed(seed)
    loras, dtype = case["loras"], TYPES[case["type"]]
    # norms around the largest allowed, 1: adapter by adapter 1/4 to 4 times it, or 3 times it over all
    count = _grad_elements(case)
    if case["per_lora"]:
        sigma = torch.exp2(4.0 * torch.rand(loras, generator=gen, device=DEVICE) - 2.0) / math.sqrt(count / loras)
    else:
        sigma = torch.full((loras,), 3.0 / math.sqrt(count), device=DEVICE)
    grads = []
    for shape in _grad_shapes(case):
        g = torch.randn(shape, generator=gen, device=DEVICE, dtype=torch.float32)
        grads.append(g.mul_(sigma.reshape([loras] + [1] * (len(shape) - 1))).to(dtype))
    # what comes out lies end to end, as the bucket that an optimizer walks
    flat = torch.empty(count, dtype=dtype, device=DEVICE)
    st = {"case": case, "grads": grads, "max_norm": 1.0, "flat": flat,
          "out": [t.reshape(g.shape) for t, g in zip(flat.split([g.numel() for g in grads]), grads)]}
    if own:
        import segmented_gather_lora_amd as sgl
        groups = loras if case["per_lora"] else 1
        st["norms"] = torch.empty(groups, dtype=torch.float32, device=DEVICE)
        # buffers of the gradients are made once, and so is the list of them
        st["held"] = sgl.LoraGradients(grads, out=st["out"])
        st["workspace"] = torch.zeros(sgl.lora_clip_gradients_workspace_bytes(st["held"], groups), dtype=torch.uint8,
                                      device=DEVICE)
    return st


def prepare(case, seed):
    return {"quantize": _prepare_quantize, "linear": _prepare_linear, "clip": _prepare_clip}[case["op"]](case, seed)


# ---------------------------------------------------------------- one pass, the library's calls

def _own_quantize(st):
    import segmented_gather_lora_amd as sgl
    sgl.lora_mx_quantize(st["x"], st["codes"], st["scales"])
    sgl.lora_mx_dequantize(st["codes"], st["scales"], st["out"])
    return st["out"]


def _own_linear(st):
    import segmented_gather_lora_amd as sgl
    sgl.lora_linear_mx(st["x"], st["codes"], st["scales"], st["w_bias"], st["a"], st["b"], st["bias"], st["buf"],
                          st["y"], st["meta"], st["scale"], st["workspace"],
                          quantize_x=st["case"]["acts"] == "mxfp4")
    if st["case"]["pass"] == "forward":
        return st["y"]
    sgl.lora_linear_mx_backward(st["dy"], st["x"], st["codes"], st["scales"], st["a"], st["b"], st["buf"],
                                   st["dbuf"], st["dx"], st["da"], st["db"], st["dbias"], st["meta"], st["scale"],
                                   st["workspace"])
    return {"y": st["y"], "dx": st["dx"], "da": st["da"], "db": st["db"],
            "dbias": [] if st["dbias"] is None else st["dbias"]}


def _own_clip(st):
    import segmented_gather_lora_amd as sgl
    sgl.lora_clip_gradients(st["held"], st["norms"], st["max_norm"], st["workspace"])
    return {"norms": st["norms"], "grads": st["flat"]}


# ---------------------------------------------------------------- one pass, plain

def _to_blocks(x):
    """Codes (two a byte, the first in the low half) and powers of two (exponent
    plus 127) of float32 rows: the power is that of the block's largest
    magnitude, less 2 (E2M1's largest power), and what it leaves is rounded to
    the nearest code, ties to the even one, and held at 6."""
    rows, cols = x.shape
    blocks = (cols + BLOCK - 1) // BLOCK
    x = torch.nn.functional.pad(x, (0, blocks * BLOCK - cols)).reshape(rows, blocks, BLOCK)
    top = x.abs().amax(2)
    power = torch.where(top > 0, torch.frexp(top)[1] - 3, torch.full_like(top, -127, dtype=torch.int32)).clamp(min=-127)
    # (two factors: 2^127 is the largest power of two in 32 bits)
    half = -power // 2
    m = torch.ldexp(torch.ldexp(x, half[..., None]), (-power - half)[..., None])
    sign = (m < 0).to(torch.uint8) << 3
    m = m.abs()
    code = torch.where(m < 2, torch.round(m * 2), torch.where(m < 4, torch.round(m) + 2, torch.round(m / 2) + 4))
    code = code.clamp(max=7).to(torch.uint8) | sign
    code = code.reshape(rows, blocks * BLOCK // 2, 2)
    scales = torch.zeros((rows, (blocks + 3) // 4 * 4), dtype=torch.uint8, device=x.device)
    scales[:, :blocks] = (power + 127).to(torch.uint8)
    return code[..., 0] | code[..., 1] << 4, scales


def _from_blocks(codes, scales, cols):
    """The numbers that codes and powers stand for, in float32."""
    table = torch.tensor(GRID + tuple(-v for v in GRID), dtype=torch.float32, device=codes.device)
    both = torch.stack((codes & 15, codes >> 4), 2).flatten(1).to(torch.int32)
    rows, wide = both.shape
    power = scales[:, :wide // BLOCK].to(torch.int32) - 127
    half = power // 2
    v = table[both].reshape(rows, wide // BLOCK, BLOCK)
    v = torch.ldexp(torch.ldexp(v, half[..., None]), (power - half)[..., None])
    return v.reshape(rows, wide)[:, :cols]


def _plain_quantize(st):
    codes, scales = _to_blocks(st["x"].float())
    return _from_blocks(codes, scales, st["case"]["cols"]).to(torch.bfloat16)


def _with_row(t):
    """t with a row of zeros after its last, for the plan's padding."""
    return torch.cat([t, t.new_zeros((1, t.shape[1]))])


def _plain_linear(st):
    """Adapters by batched products over the present ones' padded tokens; the
    comprehensions go over the slices, whose widths differ."""
    plan, present, scale, widths = st["plan"], st["present"], st["scale"], st["widths"]
    x = st["x"].float()
    w = _from_blocks(st["codes"], st["scales"], x.shape[1]).contiguous()
    seen = x if st["case"]["acts"] == "bf16" else _from_blocks(*_to_blocks(x), x.shape[1]).contiguous()
    y = _with_row(seen @ w.t())
    if st["w_bias"] is not None:
        y += st["w_bias"].float()
    a = [t[present].float() for t in st["a"]]
    b = [t[present].float() for t in st["b"]]
    xp = _with_row(x)[plan]
    s = [torch.bmm(xp, t.transpose(1, 2).contiguous()) * scale for t in a]
    delta = torch.cat([torch.bmm(u, t.transpose(1, 2).contiguous()) for u, t in zip(s, b)], 2)
    if st["bias"] is not None:
        delta += torch.cat([t[present].float() for t in st["bias"]], 1)[:, None]
    y.index_add_(0, plan.flatten(), delta.flatten(0, 1))
    y = y[:-1].to(torch.bfloat16)
    if st["case"]["pass"] == "forward":
        return y
    dy = st["dy"].float()
    dyp = _with_row(dy)[plan].split(widths, 2)
    u = [torch.bmm(d.contiguous(), t) * scale for d, t in zip(dyp, b)]
    dx = _with_row(dy @ w)
    dx.index_add_(0, plan.flatten(), sum(torch.bmm(v, t) for v, t in zip(u, a)).flatten(0, 1))
    da = [torch.zeros_like(t).index_copy_(0, present, torch.bmm(v.transpose(1, 2).contiguous(), xp).to(t.dtype))
          for v, t in zip(u, st["a"])]
    db = [torch.zeros_like(t).index_copy_(0, present, torch.bmm(d.transpose(1, 2).contiguous(), v).to(t.dtype))
          for d, v, t in zip(dyp, s, st["b"])]
    dbias = [] if st["bias"] is None else [
        torch.zeros_like(t).index_copy_(0, present, d.sum(1).to(t.dtype)) for d, t in zip(dyp, st["bias"])]
    return {"y": y, "dx": dx[:-1].to(torch.bfloat16), "da": da, "db": db, "dbias": dbias}


def _plain_clip(st):
    """A sum of squares a tensor (and adapter), and all of them together."""
    case, grads = st["case"], st["grads"]
    groups = case["loras"] if case["per_lora"] else 1
    squares = [t.reshape(groups, -1).float().square().sum(1, dtype=torch.float64) for t in grads]
    norms = torch.stack(squares).sum(0).sqrt()
    factor = torch.clamp(st["max_norm"] / (norms + 1e-6), max=1.0).float()
    for t, o in zip(grads, st["out"]):
        o.copy_((t.reshape(groups, -1).float() * factor[:, None]).reshape(t.shape))
    return {"norms": norms.float(), "grads": st["flat"]}


def run(state):
    forms = ({"quantize": _own_quantize, "linear": _own_linear, "clip": _own_clip} if own else
             {"quantize": _plain_quantize, "linear": _plain_linear, "clip": _plain_clip})
    return forms[state["case"]["op"]](state)


# ---------------------------------------------------------------- work

def work(case):
    """Each input read once and each output written once (codes and powers, too,
    between the two calls that make and read them); multiplications and
    additions of the products (of an adapter: its own tokens only)."""
    if case["op"] == "quantize":
        elements, size = float(case["rows"]) * case["cols"], 2 if case["type"] == "bf16" else 4
        return {"bytes": elements * (size + 2 * (0.5 + 1 / BLOCK) + 2), "flops": 2 * elements}
    if case["op"] == "clip":
        elements, size = float(_grad_elements(case)), 2 if case["type"] == "bf16" else 4
        return {"bytes": 2 * elements * size, "flops": 3 * elements}
    n, hidden = float(case["tokens"]), case["hidden"]
    train = case["pass"] == "train"
    widths, rank, loras = _widths(case), case["rank"], case["loras"]
    out = sum(widths)
    live = n * (1 - case["none"])
    picks = live if case["ids"] == "uniform" else math.ceil(n / (512 if case["ids"] == "runs" else 256))
    present = min(loras, picks) if case["ids"] == "dealt" else loras * (1 - (1 - 1 / loras) ** picks)
    adapters = 2.0 * present * rank * (len(widths) * hidden + out)
    moved = 2 * n * hidden + (0.5 + 1 / BLOCK) * out * hidden + 2 * n * out + adapters + 4 * n
    flops = 2 * n * hidden * out + 2 * live * rank * (len(widths) * hidden + out)
    if case["bias"]:
        moved += 2 * out + 2 * present * out
    if train:
        # dy in, dx out, the gradients of every adapter out
        moved += 2 * n * out + 2 * n * hidden + 2.0 * loras * rank * (len(widths) * hidden + out)
        moved += 2 * loras * out if case["bias"] else 0
        flops += 2 * n * hidden * out + 4 * live * rank * (len(widths) * hidden + out)
    return {"bytes": moved, "flops": flops}


# ---------------------------------------------------------------- in 64 bits

def _nearest(x):
    """Rows of x as their blocks' codes hold them, in 64 bits: every number to
    the nearest of the grid times the block's power, by the grid's midpoints."""
    grid = torch.tensor(GRID, dtype=torch.float64, device=x.device)
    mid = (grid[1:] + grid[:-1]) / 2
    out = torch.empty_like(x)
    for lo in range(0, x.shape[1], BLOCK):
        part = x[:, lo:lo + BLOCK]
        top = part.abs().amax(1, keepdim=True)
        power = torch.floor(torch.log2(torch.where(top > 0, top, 1.0))) - 2.0
        unit = torch.exp2(torch.clamp(power, min=-127.0))
        m = part.abs() / unit
        # a midpoint goes to the neighbour of even code: up from an odd one
        at = torch.searchsorted(mid, m.contiguous())
        up = (at < 7) & (m == mid[at.clamp(max=6)]) & (at % 2 == 1)
        out[:, lo:lo + BLOCK] = torch.sign(part) * grid[(at + up).clamp(max=7)] * unit
    return out


def _held(codes, scales, cols):
    """The numbers that codes stand for, from their bits: sign, two bits of
    exponent, one of mantissa."""
    out = torch.empty((codes.shape[0], cols), dtype=torch.float64, device=codes.device)
    unit = torch.exp2(scales.double() - 127.0)
    for half in (0, 1):
        c = (codes >> 4 * half & 15).long()[:, :cols // 2]
        e, m = c >> 1 & 3, (c & 1).double()
        v = torch.where(e > 0, torch.exp2(e.double() - 1.0) * (1.0 + m / 2), m / 2)
        of = torch.arange(half, cols, 2, device=codes.device) // BLOCK
        out[:, half::2] = torch.where(c >= 8, -v, v) * unit[:, of]
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "quantize":
        return _nearest(st["x"].double())
    if case["op"] == "clip":
        groups = case["loras"] if case["per_lora"] else 1
        total = torch.zeros(groups, dtype=torch.float64, device=DEVICE)
        for t in st["grads"]:
            for g in range(groups):
                v = t.reshape(groups, -1)[g].double()
                total[g] += torch.dot(v, v)
        norms = total.sqrt()
        factor = torch.where(norms + 1e-6 > st["max_norm"], st["max_norm"] / (norms + 1e-6), torch.ones_like(norms))
        return {"norms": norms,
                "grads": torch.cat([(t.reshape(groups, -1).double() * factor[:, None]).flatten() for t in st["grads"]])}
    ids = st["ids"].cpu()
    train = case["pass"] == "train"
    x = st["x"].double()
    w = _held(st["codes"], st["scales"], case["hidden"])
    y = (x if case["acts"] == "bf16" else _nearest(x)) @ w.t()
    if st["w_bias"] is not None:
        y += st["w_bias"].double()
    if train:
        dy = st["dy"].double()
        dx = dy @ w
        da = [torch.zeros(t.shape, dtype=torch.float64, device=DEVICE) for t in st["a"]]
        db = [torch.zeros(t.shape, dtype=torch.float64, device=DEVICE) for t in st["b"]]
        dbias = [] if st["bias"] is None else [torch.zeros(t.shape, dtype=torch.float64, device=DEVICE)
                                               for t in st["bias"]]
    for m in np.unique(ids.numpy()):
        if m < 0:
            continue
        rows = torch.nonzero(ids == int(m)).flatten().to(DEVICE)
        col = 0
        for i, width in enumerate(st["widths"]):
            cols = slice(col, col + width)
            a, b = st["a"][i][m].double(), st["b"][i][m].double()
            s = st["scale"] * (x[rows] @ a.t())
            add = s @ b.t()
            if st["bias"] is not None:
                add += st["bias"][i][m].double()
            y[rows, cols] += add
            if train:
                d = dy[rows, cols]
                u = st["scale"] * (d @ b)
                dx[rows] += u @ a
                da[i][m] = u.t() @ x[rows]
                db[i][m] = d.t() @ s
                if dbias:
                    dbias[i][m] = d.sum(0)
            col += width
    if not train:
        return y
    return {"y": y, "dx": dx, "da": da, "db": db, "dbias": dbias}
