"""Measured cases of the operators that serve a compressed model in 4 bits and train it on tokens:
products with 4-bit weights and group scales, and the softmax cross entropy through a model's output
matrix, without its logits kept, with its gradient.

``run`` computes a case in its plain form, elementary torch operations in 32 bits (64 where 32
lose what matters), or, with ``own`` set, through the package's entry points.  ``exact`` gives the
same outputs from the definitions in 64 bits."""

import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # one token through an attention projection while a model answers
        {"name": "grouped 1 x 2560 x 2560", "op": "grouped", "tokens": 1, "n": 2560, "m": 2560, "group": 128, "x": "bf16", "s": "bf16", "offset": False},
        # one token through an MLP's down projection, small groups with offsets
        {"name": "grouped 1 x 9728 x 2560", "op": "grouped", "tokens": 1, "n": 9728, "m": 2560, "group": 32, "x": "f16", "s": "f16", "offset": True},
        # a few tokens in fp32, no size a multiple of anything
        {"name": "grouped 7 x 1021 x 2051", "op": "grouped", "tokens": 7, "n": 1021, "m": 2051, "group": 64, "x": "f32", "s": "f32", "offset": True},
        # a batch of answers through an MLP's up projection
        {"name": "grouped 16 x 2560 x 9728", "op": "grouped", "tokens": 16, "n": 2560, "m": 9728, "group": 128, "x": "bf16", "s": "f32", "offset": False},
        # a larger batch, or a short prompt
        {"name": "grouped 100 x 2560 x 9728", "op": "grouped", "tokens": 100, "n": 2560, "m": 9728, "group": 64, "x": "bf16", "s": "bf16", "offset": True},
        # a long prompt
        {"name": "grouped 2048 x 2560 x 9728", "op": "grouped", "tokens": 2048, "n": 2560, "m": 9728, "group": 128, "x": "bf16", "s": "bf16", "offset": False},
        # the loss of one token, as in scoring an answer
        {"name": "token loss 1 x 1024 x 32768", "op": "token", "rows": 1, "n": 1024, "vocab": 32768, "x": "bf16", "kind": "loss", "dW": False, "padded": 0.0},
        # a ragged evaluation batch
        {"name": "token loss 300 x 2560 x 50021", "op": "token", "rows": 300, "n": 2560, "vocab": 50021, "x": "f16", "kind": "loss", "dW": False, "padded": 0.1},
        # a small step in fp32, odd sizes
        {"name": "token step 65 x 777 x 10007", "op": "token", "rows": 65, "n": 777, "vocab": 10007, "x": "f32", "kind": "step", "dW": True, "padded": 0.1},
        # a step of repair: the output matrix is fixed, the gradient goes to what lies below
        {"name": "token step 2048 x 2560 x 32768", "op": "token", "rows": 2048, "n": 2560, "vocab": 32768, "x": "bf16", "kind": "step", "dW": False, "padded": 0.1},
        # an evaluation of many tokens over a large vocabulary
        {"name": "token loss 4096 x 2560 x 131072", "op": "token", "rows": 4096, "n": 2560, "vocab": 131072, "x": "bf16", "kind": "loss", "dW": False, "padded": 0.0},
        # the whole backward pass of a training batch over a large vocabulary
        {"name": "token grad 2048 x 2560 x 131072", "op": "token", "rows": 2048, "n": 2560, "vocab": 131072, "x": "bf16", "kind": "grad", "dW": True, "padded": 0.0},
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    if rng.random() < 0.5:
        t, n, m = _log(rng, 1, 2048), _log(rng, 48, 9728), _log(rng, 48, 9728)
        t = max(1, min(t, 2048 * 2560 * 9728 // (n * m)))
        return {"op": "grouped", "tokens": t, "n": n, "m": m, "group": rng.choice([32, 64, 128]), "x": rng.choice(["bf16", "f16", "f32"]),
                "s": rng.choice(["bf16", "f16", "f32"]), "offset": rng.choice([False, True])}
    x, kind = rng.choice(["bf16", "bf16", "f16", "f32"]), rng.choice(["loss", "step", "grad"])
    n, v = _log(rng, 48, 4096), _log(rng, 1000, 131072)
    if rng.random() < 0.5:  # rows that are whole in 16 bytes, as most models' are
        n = (n + 7) // 8 * 8
    # a type of 32 bits has a sixteenth of the rate
    most = 2048 * 2560 * 131072 // (16 if x == "f32" else 1)
    return {"op": "token", "rows": max(1, min(_log(rng, 1, 4096), most // (n * v))), "n": n, "vocab": v, "x": x, "kind": kind,
            "dW": kind != "loss" and rng.choice([False, True]), "padded": rng.choice([0.0, 0.1, 0.5])}


def _grouped_state(case, g):
    n, m, group = case["n"], case["m"], case["group"]
    groups = (n + group - 1) // group
    # a heavy-tailed weight matrix: a normal one over the root of a mean of four squares
    w = torch.zeros((m, groups * group), device="cuda")
    w[:, :n] = torch.randn((m, n), generator=g, device="cuda")
    d = torch.zeros_like(w)
    for _ in range(4):
        d += torch.randn(w.shape, generator=g, device="cuda").square_()
    w = w.mul_(0.02 / math.sqrt(2.0)).div_(d.mul_(0.25).sqrt_()).view(m, groups, group)
    if case["offset"]:
        lo, hi = w.amin(2, keepdim=True), w.amax(2, keepdim=True)
        step = (hi - lo) / 15
        code = torch.round((w - lo) / step) - 8
        offset = (lo + 8 * step)[:, :, 0].to(TYPES[case["s"]]).contiguous()
    else:
        step = w.abs().amax(2, keepdim=True) / 7
        code, offset = torch.round(w / step), None
    code = code.view(m, -1).to(torch.int64)
    code[:, n:] = 0
    # eight codes a word, the first in the lowest bits, two's complement
    word = ((code & 15).view(m, -1, 8) << (4 * torch.arange(8, device="cuda"))).sum(2)
    # activations: normal, with one channel in 300 twenty times larger
    x = torch.randn((case["tokens"], n), generator=g, device="cuda")
    x *= torch.where(torch.rand((n,), generator=g, device="cuda") < 1 / 300, 20.0, 1.0)
    return {"op": "grouped", "Q": torch.where(word >= 2**31, word - 2**32, word).to(torch.int32), "scale": step[:, :, 0].to(TYPES[case["s"]]).contiguous(),
            "offset": offset, "group": group, "X": x.to(TYPES[case["x"]])}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "grouped":
        return _grouped_state(case, g)
    rows, n, v, t = case["rows"], case["n"], case["vocab"], TYPES[case["x"]]
    w = torch.randn((v, n), generator=g, device="cuda").mul_(n**-0.5).to(t)
    target = torch.randint(0, v, (rows,), generator=g, device="cuda")
    # a trained model's hidden rows: near the target's row for some tokens, far from it for others
    sure = 12.0 * torch.rand((rows, 1), generator=g, device="cuda")
    x = (torch.randn((rows, n), generator=g, device="cuda").mul_(1.5) + sure * w[target].float()).to(t)
    keep = torch.rand((rows,), generator=g, device="cuda") >= case["padded"]
    keep[0] = True
    # a mean over the kept tokens; half-precision gradients are scaled up, as loss scaling does
    weight = keep.float() / keep.sum() * (1.0 if case["x"] != "f16" else 65536.0)
    s = {"op": "token", "kind": case["kind"], "dW": case["dW"], "X": x, "W": w, "target": torch.where(keep, target, -100), "weight": weight}
    if case["kind"] == "grad":  # the forward pass's statistics: the row's largest logit and sum of exp(z - largest)
        s["stats"] = torch.empty((rows, 2), device="cuda")
        for i in range(0, rows, 256):
            z = x[i:i + 256].float() @ w.float().t()
            top = z.amax(1, keepdim=True)
            s["stats"][i:i + 256] = torch.cat([top, z.sub_(top).exp_().sum(1, keepdim=True, dtype=torch.float64).float()], 1) * keep[i:i + 256, None]
    return s


def run(s):
    return _grouped(s) if s["op"] == "grouped" else _token(s)


def _package():
    import expanded_rank_matrix_amd as erm

    return erm


def _grouped(s):
    x, scale, group = s["X"], s["scale"], s["group"]
    if own:
        return _package().apply_grouped(s["Q"], scale, x, offset=s["offset"], group=group)
    m, groups = scale.shape
    code = (s["Q"][:, :, None] >> (4 * torch.arange(8, device=x.device, dtype=torch.int32))) & 15
    w = (code - 16 * (code >> 3)).view(m, groups, group).float() * scale.float()[:, :, None]
    if s["offset"] is not None:
        w = w + s["offset"].float()[:, :, None]
    return (x.float() @ w.view(m, -1)[:, :x.shape[1]].t()).to(x.dtype)


def _token(s):
    x, w, target, weight = s["X"], s["W"], s["target"], s["weight"]
    if own:
        erm = _package()
        if s["kind"] == "grad":
            return erm.token_grad(x, w, s["stats"], target, grad_loss=weight, need_dW=s["dW"])
        return erm.token_loss(x, w, target, weight=weight, grad=s["kind"] == "step", need_dW=s["dW"])
    kept = ((weight != 0) & (target >= 0) & (target < w.shape[0]))[:, None]
    at = torch.where(kept, target[:, None], 0)
    xf, wf = torch.where(kept, x.float(), 0.0), w.float()
    z = xf @ wf.t()
    if s["kind"] == "grad":
        top, total = s["stats"][:, :1], s["stats"][:, 1:]
        q = z.sub_(top).exp_().div_(torch.where(kept, total, 1.0))
        out = ()
    else:
        top = z.amax(1, keepdim=True)
        zt = z.gather(1, at)
        q = z.sub_(top).exp_()
        total = q.sum(1, keepdim=True, dtype=torch.float64)
        loss = (top.double() - zt.double() + total.log())[:, 0] * weight
        out = (torch.where(kept[:, 0], loss, 0.0).float(), torch.where(kept, torch.cat([top, total.float()], 1), 0.0))
        if s["kind"] == "loss":
            return out
        q = q.div_(total.float())
    d = q.scatter_add_(1, at, torch.full_like(top, -1.0)).mul_(torch.where(kept, weight[:, None], 0.0))
    return (*out, (d @ wf).to(x.dtype), (d.t() @ xf).to(w.dtype) if s["dW"] else None)


def work(case):
    if case["op"] == "grouped":
        t, n, m, groups = case["tokens"], case["n"], case["m"], (case["n"] + case["group"] - 1) // case["group"]
        scales = m * groups * SIZE[case["s"]] * (2 if case["offset"] else 1)
        return {"bytes": m * groups * case["group"] // 2 + scales + t * (n + m) * SIZE[case["x"]], "flops": 2 * t * n * m}
    # padded rows are not read, their gradient is written; a product for the logits and one for each gradient
    r, n, v, e = case["rows"], case["n"], case["vocab"], SIZE[case["x"]]
    kept = round(r * (1 - case["padded"]))
    products, written = 1, 12 * r
    if case["kind"] != "loss":
        products, written = 2 + case["dW"], written + (r + (v if case["dW"] else 0)) * n * e
    return {"bytes": (kept + v) * n * e + 12 * r + written, "flops": 2 * products * kept * n * v}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "grouped":
        m, n, group = case["m"], case["n"], case["group"]
        w = torch.empty((m, s["Q"].shape[1], 8), dtype=torch.float64, device="cuda")
        for e in range(8):
            # the code's four bits moved to the word's top and back down with their sign
            w[:, :, e] = (s["Q"] << (28 - 4 * e)) >> 28
        w = w.view(m, -1, group).mul_(s["scale"].double().unsqueeze(2))
        if s["offset"] is not None:
            w.add_(s["offset"].double().unsqueeze(2))
        return torch.mm(s["X"].double(), w.view(m, -1)[:, :n].t().contiguous())
    rows, n, v = case["rows"], case["n"], case["vocab"]
    w = s["W"].double()
    wt = w.t().contiguous()
    loss = torch.zeros(rows, dtype=torch.float64, device="cuda")
    stats = torch.zeros((rows, 2), dtype=torch.float64, device="cuda")
    grads = case["kind"] != "loss"
    dx = torch.zeros((rows, n), dtype=torch.float64, device="cuda") if grads else None
    dw = torch.zeros((v, n), dtype=torch.float64, device="cuda") if case["dW"] else None
    counted = torch.nonzero((s["weight"] != 0) & (s["target"] != -100))[:, 0]
    for at in counted.split(256):  # 64-bit rows a few at a time
        x, t, g = s["X"][at].double(), s["target"][at], s["weight"][at].double()
        z = torch.mm(x, wt)
        lse = torch.logsumexp(z, dim=1)
        own_logit = torch.gather(z, 1, t[:, None])[:, 0]
        largest = z.max(dim=1).values
        loss[at] = g * (lse - own_logit)
        stats[at] = torch.stack([largest, torch.exp(lse - largest)], dim=1)
        if grads:
            d = torch.exp(z - lse[:, None])
            d[torch.arange(len(at), device="cuda"), t] -= 1.0
            d *= g[:, None]
            dx[at] = torch.mm(d, w)
            if dw is not None:
                dw += torch.mm(d.t().contiguous(), x)
    return {"loss": (loss, stats), "step": (loss, stats, dx, dw), "grad": (dx, dw)}[case["kind"]]
