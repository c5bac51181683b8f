"""The two operators beside the multi-LoRA path, as cases that can be timed.

``linear``: a projection that every request shares (a frozen bf16 matrix) with
the low-rank adapters of many requests added in the same product; its forward
pass (``pass: "forward"``, serving) and a training step of the adapters
(``pass: "train"``: forward, then the gradients of the input, the adapters and
their bias).

``loss``: softmax cross entropy of hidden states against a vocabulary matrix,
in pieces of the vocabulary, without the logits in memory: the per-token loss
(``pass: "score"``) and a training step (``pass: "train"``: the loss, then the
gradients of the hidden states and, where the head trains, of the matrix).

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


# ---------------------------------------------------------------- cases

def _linear(name, step, tokens, hidden, slices, rank, loras, ids, none, bias):
    return {"name": name, "op": "linear", "pass": step, "tokens": tokens, "hidden": hidden,
            "slices": ",".join(str(w) for w in slices), "rank": rank, "loras": loras, "ids": ids,
            "none": none, "bias": bias}


def _loss(name, step, tokens, hidden, vocab, ignored, head):
    return {"name": name, "op": "loss", "pass": step, "tokens": tokens, "hidden": hidden, "vocab": vocab,
            "ignored": ignored, "head": head}


def listed():
    return [
        # one request's next token through a q/k/v projection: latency alone
        _linear("linear one token", "forward", 1, 4096, (4096, 1024, 1024), 16, 32, "uniform", 0.0, False),
        # a decode step of 256 requests over 32 adapters
        _linear("linear decode", "forward", 256, 4096, (4096, 1024, 1024), 16, 32, "uniform", 0.10, False),
        # prompts of 512 tokens each, with the shared and the adapters' biases
        _linear("linear prefill", "forward", 8192, 4096, (4096, 1024, 1024), 64, 8, "runs", 0.0, True),
        # nothing a multiple of a tile, a slice of 8 columns, a quarter without an adapter
        _linear("linear odd", "forward", 1003, 1032, (264, 8, 520), 24, 9, "uniform", 0.25, True),
        # the largest mixed batch: 16384 interleaved tokens of 128 adapters of rank 128
        _linear("linear train mixed", "train", 16384, 8192, (8192, 1024, 1024), 128, 128, "uniform", 0.20, False),
        # gate and up projections, sequences of 256 tokens dealt to 16 adapters
        _linear("linear train gate up", "train", 4096, 4096, (14336, 14336), 32, 16, "dealt", 0.0, False),
        # a small ragged step with biases
        _linear("linear train odd", "train", 517, 520, (136, 72), 8, 5, "uniform", 0.20, True),
        # the sampled tokens' log-probabilities of one small decode step
        _loss("score 16", "score", 16, 4096, 128256, 0.0, False),
        # 256 prompts' positions over the whole vocabulary
        _loss("score 256", "score", 256, 4096, 128256, 0.10, False),
        # adapters train, the head is frozen: gradient of the hidden states only
        _loss("loss train frozen head", "train", 2048, 4096, 128256, 0.25, False),
        # the head trains too
        _loss("loss train head", "train", 4096, 4096, 128256, 0.10, True),
        # an odd vocabulary and few tokens
        _loss("loss train odd", "train", 301, 264, 5003, 0.20, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    """One more case of the ranges: tokens 1..16384, widths in steps of 8 (the
    library's rows are 16-byte aligned), any vocabulary up to 131072."""
    most = max(work(c)["flops"] for c in listed())
    while True:
        if rng.random() < 0.55:
            tokens, hidden = _log(rng, 1, 16384), 8 * _log(rng, 16, 1024)
            slices = [8 * _log(rng, 1, 1024) for _ in range(rng.choice((1, 1, 2, 3)))]
            case = _linear("", rng.choice(("forward", "train")), tokens, hidden, slices, 8 * rng.randint(1, 16),
                           _log(rng, 1, 128), rng.choice(("uniform", "runs", "dealt")),
                           rng.choice((0.0, 0.1, 0.3)), rng.random() < 0.4)
        else:
            case = _loss("", rng.choice(("score", "train")), _log(rng, 1, 8192), 8 * _log(rng, 16, 640),
                         _log(rng, 100, 131072), rng.choice((0.0, 0.1, 0.4)), rng.random() < 0.5)
        del case["name"]
        if work(case)["flops"] <= most and _bytes_held(case) < 12e9:
            return case


def _bytes_held(case):
    """Bytes of the largest things that the plain form holds in 32 bits."""
    if case["op"] == "loss":
        return 12.0 * case["tokens"] * case["vocab"] + 8.0 * case["vocab"] * case["hidden"]
    wide = sum(_widths(case)) + case["hidden"]
    return 16.0 * case["tokens"] * wide + 8.0 * case["loras"] * case["rank"] * wide * len(_widths(case))


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
    st = {"case": case, "ids": ids.to(DEVICE), "present": present.to(DEVICE), "plan": plan.to(DEVICE),
          "scale": 2.0 / math.sqrt(rank), "widths": widths,
          "x": _normal(gen, (n, hidden)), "w": _normal(gen, (out, hidden), SIGMA_W),
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
        st["workspace"] = torch.zeros(sgl.lora_linear_workspace_bytes(n, loras, hidden, widths, rank, train),
                                      dtype=torch.uint8, device=DEVICE)
        if train:
            st["dbuf"] = torch.empty_like(st["buf"])
            st["dx"] = torch.empty_like(st["x"])
            st["da"] = [torch.empty_like(t) for t in st["a"]]
            st["db"] = [torch.empty_like(t) for t in st["b"]]
            st["dbias"] = None if st["bias"] is None else [torch.empty_like(t) for t in st["bias"]]
    return st


def _prepare_loss(case, seed):
    gen = torch.Generator(DEVICE).manual_seed(seed)
    n, hidden, vocab = case["tokens"], case["hidden"], case["vocab"]
    w = _normal(gen, (vocab, hidden), SIGMA_W)
    true = torch.randint(0, vocab, (n,), generator=gen, device=DEVICE)
    # a model that has learned something: the target's logit is raised by 0 to 12
    sure = 12.0 * torch.rand((n, 1), generator=gen, device=DEVICE)
    rows = w[true].float()
    x = torch.randn((n, hidden), generator=gen, device=DEVICE)
    x = (x + sure * rows / (rows * rows).sum(1, keepdim=True)).to(torch.bfloat16)
    targets = true.to(torch.int32)
    ignored = int(round(case["ignored"] * n))
    if ignored:
        targets[torch.randperm(n, generator=gen, device=DEVICE)[:ignored]] = -1
    st = {"case": case, "x": x, "w": w, "targets": targets}
    if case["pass"] == "train":
        # the mean over the tokens that count
        st["dloss"] = torch.full((n,), 1.0 / max(1, n - ignored), dtype=torch.float32, device=DEVICE)
    if own:
        import segmented_gather_lora_amd as sgl
        train = case["pass"] == "train"
        st["loss"] = torch.empty(n, dtype=torch.float32, device=DEVICE)
        st["lse"] = torch.empty(n, dtype=torch.float32, device=DEVICE)
        st["workspace"] = torch.zeros(sgl.lora_cross_entropy_workspace_bytes(n, hidden, vocab, train),
                                      dtype=torch.uint8, device=DEVICE)
        if train:
            st["dx"] = torch.empty_like(x)
            st["dw"] = torch.empty_like(w) if case["head"] else None
    return st


def prepare(case, seed):
    return (_prepare_linear if case["op"] == "linear" else _prepare_loss)(case, seed)


# ---------------------------------------------------------------- one pass

def _own_linear(st):
    import segmented_gather_lora_amd as sgl
    sgl.lora_linear(st["x"], st["w"], st["w_bias"], st["a"], st["b"], st["bias"], st["buf"], st["y"], st["meta"],
                    st["scale"], st["workspace"])
    if st["case"]["pass"] == "forward":
        return st["y"]
    sgl.lora_linear_backward(st["dy"], st["x"], st["w"], st["a"], st["b"], st["buf"], st["dbuf"], st["dx"], st["da"],
                             st["db"], st["dbias"], st["meta"], st["scale"], st["workspace"])
    return {"y": st["y"], "dx": st["dx"], "da": st["da"], "db": st["db"],
            "dbias": [] if st["dbias"] is None else st["dbias"]}


def _own_loss(st):
    import segmented_gather_lora_amd as sgl
    sgl.lora_cross_entropy(st["x"], st["w"], st["targets"], st["loss"], st["lse"], st["workspace"])
    if st["case"]["pass"] == "score":
        return {"loss": st["loss"], "lse": st["lse"]}
    sgl.lora_cross_entropy_backward(st["x"], st["w"], st["targets"], st["lse"], st["dloss"], st["dx"], st["dw"],
                                    st["workspace"])
    return {"loss": st["loss"], "lse": st["lse"], "dx": st["dx"], "dw": [] if st["dw"] is None else [st["dw"]]}


def _with_row(t):
    """t with a row of zeros after its last, for the plan's padding."""
    return torch.cat([t, t.new_zeros((1, t.shape[1]))])


def _plain_linear(st):
    """Adapters by batched products over the present ones' padded tokens; the
    comprehensions go over the slices, whose widths differ."""
    plan, present, scale, widths = st["plan"], st["present"], st["scale"], st["widths"]
    x = st["x"].float()
    y = _with_row(x @ st["w"].float().t())
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
    dx = _with_row(dy @ st["w"].float())
    dx.index_add_(0, plan.flatten(), sum(torch.bmm(v, t) for v, t in zip(u, a)).flatten(0, 1))
    da = [torch.zeros_like(t).index_copy_(0, present, torch.bmm(v.transpose(1, 2).contiguous(), xp).to(t.dtype))
          for v, t in zip(u, st["a"])]
    db = [torch.zeros_like(t).index_copy_(0, present, torch.bmm(d.transpose(1, 2).contiguous(), v).to(t.dtype))
          for d, v, t in zip(dyp, s, st["b"])]
    dbias = [] if st["bias"] is None else [
        torch.zeros_like(t).index_copy_(0, present, d.sum(1).to(t.dtype)) for d, t in zip(dyp, st["bias"])]
    return {"y": y, "dx": dx[:-1].to(torch.bfloat16), "da": da, "db": db, "dbias": dbias}


def _plain_loss(st):
    x, w = st["x"].float(), st["w"].float()
    targets = st["targets"].long()
    counts = targets >= 0
    at = targets.clamp(min=0)[:, None]
    logits = x @ w.t()
    top = logits.max(1, keepdim=True).values
    terms = (logits - top).exp()
    total = terms.sum(1, keepdim=True)
    lse = (top + total.log())[:, 0]
    loss = torch.where(counts, lse - logits.gather(1, at)[:, 0], torch.zeros_like(lse))
    if st["case"]["pass"] == "score":
        return {"loss": loss, "lse": lse}
    g = terms / total
    g.scatter_add_(1, at, torch.full_like(lse, -1.0)[:, None])
    g *= torch.where(counts, st["dloss"], torch.zeros_like(lse))[:, None]
    return {"loss": loss, "lse": lse, "dx": (g @ w).to(torch.bfloat16),
            "dw": [(g.t() @ x).to(torch.bfloat16)] if st["case"]["head"] else []}


def run(state):
    if own:
        return (_own_linear if state["case"]["op"] == "linear" else _own_loss)(state)
    return (_plain_linear if state["case"]["op"] == "linear" else _plain_loss)(state)


# ---------------------------------------------------------------- work

def work(case):
    """Each input read once and each output written once; multiplications and
    additions of the products (of an adapter: its own tokens only)."""
    n, hidden = float(case["tokens"]), case["hidden"]
    train = case["pass"] == "train"
    if case["op"] == "loss":
        vocab = case["vocab"]
        products = 1 + train + (train and case["head"])
        moved = 2 * (n + vocab) * hidden + 12 * n
        if train:
            moved += 2 * n * hidden + (2.0 * vocab * hidden if case["head"] else 0)
        return {"bytes": moved, "flops": 2.0 * n * vocab * hidden * products}
    widths, rank, loras = _widths(case), case["rank"], case["loras"]
    out = sum(widths)
    live = n * (1 - case["none"])
    picks = live if case["ids"] == "uniform" else math.ceil(n / (512 if case["ids"] == "runs" else 256))
    present = min(loras, picks) if case["ids"] == "dealt" else loras * (1 - (1 - 1 / loras) ** picks)
    adapters = 2.0 * present * rank * (len(widths) * hidden + out)
    moved = 2 * (n + out) * hidden + 2 * n * out + adapters + 4 * n
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

def exact(case, seed):
    st = prepare(case, seed)
    x, w = st["x"].double(), st["w"].double()
    if case["op"] == "loss":
        n = case["tokens"]
        targets = st["targets"].cpu().numpy()
        keep = np.flatnonzero(targets >= 0)
        loss = torch.zeros(n, dtype=torch.float64, device=DEVICE)
        lse = torch.zeros(n, dtype=torch.float64, device=DEVICE)
        dx = torch.zeros_like(x)
        dw = torch.zeros_like(w) if case["pass"] == "train" and case["head"] else None
        step = 512
        for lo in range(0, n, step):
            z = torch.matmul(x[lo:lo + step], w.t())
            lse[lo:lo + step] = torch.logsumexp(z, 1)
            rows = torch.from_numpy(keep[(keep >= lo) & (keep < lo + step)]).to(DEVICE)
            t = st["targets"][rows].long()
            loss[rows] = lse[rows] - z[rows - lo, t]
            if case["pass"] == "train":
                p = torch.zeros_like(z)
                p[rows - lo] = torch.exp(z[rows - lo] - lse[rows, None])
                p[rows - lo, t] -= 1.0
                p *= st["dloss"][lo:lo + step, None].double()
                dx[lo:lo + step] = p @ w
                if dw is not None:
                    dw += p.t() @ x[lo:lo + step]
        if case["pass"] == "score":
            return {"loss": loss, "lse": lse}
        return {"loss": loss, "lse": lse, "dx": dx, "dw": [] if dw is None else [dw]}
    ids = st["ids"].cpu()
    train = case["pass"] == "train"
    y = x @ w.t()
    if st["w_bias"] is not None:
        y += st["w_bias"].double()
    if train:
        dy = st["dy"].double()
        dx = dy @ w
        da = [torch.zeros(t.shape, dtype=torch.float64, device=DEVICE) for t in st["a"]]
        db = [torch.zeros(t.shape, dtype=torch.float64, device=DEVICE) for t in st["b"]]
        dbias = [] if st["bias"] is None else [torch.zeros(t.shape, dtype=torch.float64, device=DEVICE)
                                               for t in st["bias"]]
    for m in sorted(set(ids.tolist()) - {-1}):
        rows = torch.nonzero(ids == m).flatten().to(DEVICE)
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
