"""Measured cases of the operators that run a compressed model and repair it: products in 8-bit
integers with scales for each token and channel, the distillation loss on a teacher's top logits
with its gradient, and the gradient of a layer held as packed ternary factors.

``run`` computes a case in its plain form, elementary torch operations in 32 bits (64 where 32
lose what matters), or, with ``own`` set, through the package's entry points.  ``exact`` gives the
same outputs from the definitions in 64 bits."""

import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "i8": torch.int8}


def listed():
    return [
        # one token through an attention projection while a model answers
        {"name": "product 1 x 2560 x 2560", "op": "product", "tokens": 1, "n": 2560, "m": 2560, "x": "bf16", "y": "bf16"},
        # a small batch of answers through an MLP's up projection
        {"name": "product 16 x 2560 x 9728", "op": "product", "tokens": 16, "n": 2560, "m": 9728, "x": "bf16", "y": "bf16"},
        # a short prompt, no size a multiple of anything
        {"name": "product 333 x 1021 x 2051", "op": "product", "tokens": 333, "n": 1021, "m": 2051, "x": "f16", "y": "f16"},
        # a prompt whose tokens were quantised once for several products
        {"name": "product 2048 x 2560 x 9728", "op": "product", "tokens": 2048, "n": 2560, "m": 9728, "x": "i8", "y": "bf16"},
        # a long prompt through an MLP's down projection, quantised on the way
        {"name": "product 4096 x 9728 x 2560", "op": "product", "tokens": 4096, "n": 9728, "m": 2560, "x": "bf16", "y": "f32"},
        # the quantisation alone, as done once for several products
        {"name": "quantize 4096 x 9728", "op": "quantize", "rows": 4096, "n": 9728, "x": "bf16"},
        # the loss alone on a small, ragged evaluation batch
        {"name": "distill 65 x 50021", "op": "distill", "rows": 65, "vocab": 50021, "top": 33, "z": "f32", "kind": "loss", "temperature": 2.0, "padded": 0.1},
        # a training step: loss and gradient in one call, one token in ten padding
        {"name": "distill step 2048 x 32768", "op": "distill", "rows": 2048, "vocab": 32768, "top": 64, "z": "bf16", "kind": "step", "temperature": 1.0, "padded": 0.1},
        # the backward pass alone over a large vocabulary
        {"name": "distill grad 2048 x 131072", "op": "distill", "rows": 2048, "vocab": 131072, "top": 128, "z": "bf16", "kind": "grad", "temperature": 1.5, "padded": 0.0},
        # one vector back through a factored attention projection
        {"name": "factors grad 1, k 7680", "op": "factors", "batch": 1, "k": 7680, "m": 2560, "n": 2560},
        # an odd small layer and batch
        {"name": "factors grad 37, k 1203", "op": "factors", "batch": 37, "k": 1203, "m": 777, "n": 1025},
        # a training batch back through a factored attention projection
        {"name": "factors grad 2048, k 7680", "op": "factors", "batch": 2048, "k": 7680, "m": 2560, "n": 2560},
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["product", "product", "product", "quantize", "distill", "distill", "factors", "factors"])
    if op == "product":
        t, n, m = _log(rng, 1, 4096), _log(rng, 48, 9728), _log(rng, 48, 9728)
        t = max(1, min(t, 4096 * 9728 * 2560 // (n * m)))
        return {"op": op, "tokens": t, "n": n, "m": m, "x": rng.choice(["bf16", "f16", "f32", "i8"]), "y": rng.choice(["bf16", "f16", "f32"])}
    if op == "quantize":
        return {"op": op, "rows": _log(rng, 1, 4096), "n": _log(rng, 48, 9728), "x": rng.choice(["bf16", "f16", "f32"])}
    if op == "distill":
        v = _log(rng, 1000, 131072)
        return {"op": op, "rows": _log(rng, 1, 2048), "vocab": v, "top": _log(rng, 1, 256), "z": rng.choice(["bf16", "f16", "f32"]),
                "kind": rng.choice(["loss", "step", "grad"]), "temperature": rng.choice([1.0, 1.5, 2.0, 4.0]), "padded": rng.choice([0.0, 0.1, 0.5])}
    k, m, n = _log(rng, 96, 7680), _log(rng, 48, 9728), _log(rng, 48, 9728)
    b = max(1, min(_log(rng, 1, 2048), 2048 * 7680 * 2560 * 3 // (k * (m + 2 * n))))
    return {"op": op, "batch": b, "k": k, "m": m, "n": n}


def _activations(rows, n, dtype, g):
    """Activations: normal, with one channel in 300 twenty times larger."""
    x = torch.randn((rows, n), generator=g, device="cuda")
    x *= torch.where(torch.rand((n,), generator=g, device="cuda") < 1 / 300, 20.0, 1.0)
    return x.to(dtype)


def _weights(rows, n, g):
    """A heavy-tailed weight matrix: a normal one over the root of a mean of four squares."""
    w = torch.randn((rows, n), generator=g, device="cuda")
    d = torch.zeros_like(w)
    for _ in range(4):
        d += torch.randn((rows, n), generator=g, device="cuda").square_()
    return w.mul_(0.02 / math.sqrt(2.0)).div_(d.mul_(0.25).sqrt_())


def _codes(k, length, zeros, g):
    """k packed ternary rows: 2-bit codes 0, 1, 3, sixteen a word, the words' last codes 0."""
    words = (length + 15) // 16
    r = torch.rand((k, words * 16), generator=g, device="cuda")
    c = torch.where(r < zeros, 0, torch.where(r < 0.5 * (1 + zeros), 1, 3)).to(torch.int64)
    c[:, length:] = 0
    w = (c.view(k, words, 16) << (2 * torch.arange(16, device="cuda"))).sum(2)
    return torch.where(w >= 2**31, w - 2**32, w).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "product":
        w = _weights(case["m"], case["n"], g)
        a = w.abs().amax(1, keepdim=True)
        s = {"W": torch.round(w / a * 127).to(torch.int8), "w_scale": (a / 127)[:, 0].contiguous(), "x_scale": None, "y": TYPES[case["y"]]}
        x = _activations(case["tokens"], case["n"], torch.float32 if case["x"] == "i8" else TYPES[case["x"]], g)
        if case["x"] == "i8":
            a = x.abs().amax(1, keepdim=True)
            s["x_scale"] = (a / 127)[:, 0].contiguous()
            x = torch.round(x / a * 127).to(torch.int8)
        return {"op": "product", "X": x, **s}
    if case["op"] == "quantize":
        return {"op": "quantize", "X": _activations(case["rows"], case["n"], TYPES[case["x"]], g)}
    if case["op"] == "distill":
        rows, v, top = case["rows"], case["vocab"], case["top"]
        t = torch.randn((rows, v), generator=g, device="cuda").mul_(3.0)
        a, index = torch.topk(t, top, dim=1)
        absent = torch.rand((rows, top), generator=g, device="cuda") < 0.02  # shorter lists end in -1
        absent[:, 0] = False
        z = t.add_(torch.randn((rows, v), generator=g, device="cuda")).to(TYPES[case["z"]])
        keep = torch.rand((rows,), generator=g, device="cuda") >= case["padded"]
        # a mean over the kept tokens; half-precision gradients are scaled up, as loss scaling does
        weight = keep.float() / keep.sum().clamp(min=1) * (1.0 if case["z"] != "f16" else 65536.0)
        s = {"op": "distill", "kind": case["kind"], "z": z, "teacher": a, "index": torch.where(absent, -1, index).to(torch.int32), "T": case["temperature"], "weight": weight}
        if case["kind"] == "grad":  # the forward pass's statistics: the row's largest logit and sum of exp((z - largest) / T)
            zf = z.float()
            top1 = zf.amax(1, keepdim=True)
            s["stats"] = torch.cat([top1, zf.sub_(top1).div_(case["temperature"]).exp_().sum(1, keepdim=True, dtype=torch.float64).float()], 1)
        return s
    k, m, n, b = case["k"], case["m"], case["n"], case["batch"]
    d = torch.randn((k,), generator=g, device="cuda").abs_().mul_(0.02)
    return {"op": "factors", "B": _codes(k, m, 0.4, g), "C": _codes(k, n, 0.4, g), "D": d, "m": m, "n": n,
            "X": _activations(b, n, torch.float32, g), "dY": torch.randn((b, m), generator=g, device="cuda").mul_(1.0 / b)}


def run(s):
    if s["op"] == "product":
        return _product(s)
    if s["op"] == "quantize":
        return _quantize(s["X"]) if not own else _package().quantize_rows(s["X"])
    if s["op"] == "distill":
        return _distill(s)
    return _factors(s)


def _package():
    import expanded_rank_matrix_amd as erm

    return erm


def _quantize(x):
    """Rows in 64 bits: a quotient next to a border between two whole numbers rounds as defined."""
    a = x.abs().amax(1, keepdim=True).double()
    q = torch.round(x.double() * 127 / torch.where(a > 0, a, 1.0))
    return q.to(torch.int8), (a / 127).float()[:, 0]


def _product(s):
    if own:
        return _package().apply_quantized(s["W"], s["w_scale"], s["X"], s["x_scale"], out_dtype=s["y"])
    q, scale = (s["X"], s["x_scale"]) if s["x_scale"] is not None else _quantize(s["X"])
    return (q.float() @ s["W"].float().t() * scale[:, None] * s["w_scale"]).to(s["y"])


def _distill(s):
    z, a, index, T, w = s["z"], s["teacher"], s["index"], s["T"], s["weight"]
    if own:
        erm = _package()
        if s["kind"] == "grad":
            return erm.distill_grad(z, s["stats"], a, index, temperature=T, grad_loss=w)
        return erm.distill_loss(z, a, index, temperature=T, weight=w, grad=s["kind"] == "step")
    kept = (w != 0)[:, None]
    valid = (index >= 0) & (index < z.shape[1])
    at = torch.where(valid, index, 0).long()
    la = torch.where(valid, a, -torch.inf) / T
    la = la - la.amax(1, keepdim=True)
    p = la.exp()
    p = p / p.sum(1, keepdim=True)
    zf = z.float()
    if s["kind"] == "grad":
        top, total = s["stats"][:, :1], s["stats"][:, 1:]
        q = zf.sub(top).div_(T).exp_().div_(total)
    else:
        top = zf.amax(1, keepdim=True)
        e = zf.sub(top).div_(T).exp_()
        total = e.sum(1, keepdim=True, dtype=torch.float64).float()
        logq = (zf.gather(1, at) - top).double() / T - total.double().log()
        logp = p.double().log()
        loss = torch.where(valid & (p > 0), p * (logp - logq), 0.0).sum(1) * (T * T * w)
        out = (torch.where(kept[:, 0], loss, 0.0).float(), torch.where(kept, torch.cat([top, total], 1), 0.0))
        if s["kind"] == "loss":
            return out
        q = e.div_(total)
    d = q.scatter_add_(1, at, -torch.where(valid, p, 0.0)).mul_((w * T)[:, None])
    d = torch.where(kept, d, 0.0).to(z.dtype)
    return d if s["kind"] == "grad" else (*out, d)


def _unpacked(words, length):
    c = (words[:, :, None] >> (2 * torch.arange(16, device=words.device, dtype=torch.int32))) & 3
    return (c - 4 * (c >> 1)).reshape(words.shape[0], -1)[:, :length].float()


def _factors(s):
    if own:
        return _package().apply_factors_grad(s["B"], s["C"], s["D"], s["m"], s["n"], s["X"], s["dY"])
    c = _unpacked(s["C"], s["n"])
    u = s["dY"] @ _unpacked(s["B"], s["m"]).t()
    t = s["X"] @ c.t()
    return (u * s["D"]) @ c, (t * u).sum(0, dtype=torch.float64).float()


def work(case):
    size = {"f32": 4, "f16": 2, "bf16": 2, "i8": 1}
    if case["op"] == "product":
        t, n, m = case["tokens"], case["n"], case["m"]
        return {"bytes": t * n * size[case["x"]] + m * n + t * m * size[case["y"]] + 4 * m + (4 * t if case["x"] == "i8" else 0), "flops": 2 * t * n * m}
    if case["op"] == "quantize":
        r, n = case["rows"], case["n"]
        return {"bytes": r * n * (size[case["x"]] + 1) + 4 * r, "flops": 3 * r * n}
    if case["op"] == "distill":
        # padding rows are not read; a gradient's are written
        r, v, e = case["rows"], case["vocab"], size[case["z"]]
        read = round(r * (1 - case["padded"])) * (v * e + 8 * case["top"])
        return {"bytes": read + (0 if case["kind"] == "loss" else r * v * e) + 16 * r, "flops": 5 * r * v}
    b, k, m, n = case["batch"], case["k"], case["m"], case["n"]
    return {"bytes": k * ((m + 15) // 16 + (n + 15) // 16) * 4 + 8 * k + 4 * b * (m + 2 * n), "flops": 2 * b * k * (m + 2 * n)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("product", "quantize"):
        x = s["X"].double()
        if s.get("x_scale") is None:
            largest = x.abs().max(dim=1).values
            q = torch.round(x / largest.clamp(min=1e-300)[:, None] * 127.0)
            if case["op"] == "quantize":
                return q.to(torch.int8), largest / 127.0
            scale = largest / 127.0
        else:
            q, scale = x, s["x_scale"].double()
        return torch.mm(q, s["W"].double().t().contiguous()) * torch.outer(scale, s["w_scale"].double())
    if case["op"] == "distill":
        T, w = case["temperature"], s["weight"].double()
        parts = [[], [], []]
        for i in range(0, case["rows"], 256):  # 64-bit rows a few at a time
            z, w_i, index = s["z"][i:i + 256].double(), w[i:i + 256], s["index"][i:i + 256].long()
            lse = torch.logsumexp(z / T, dim=1, keepdim=True)
            some = index != -1
            a = s["teacher"][i:i + 256].double().masked_fill(~some, -math.inf) / T
            p = torch.softmax(a, dim=1)
            entropy = -torch.special.entr(p).sum(1)
            cross = (p * (torch.gather(z, 1, index.clamp(min=0)) / T - lse)).masked_fill(~some, 0.0).sum(1)
            largest = z.max(dim=1).values
            parts[0].append(w_i * T**2 * (entropy - cross))
            parts[1].append(torch.stack([largest, torch.exp(lse[:, 0] - largest / T)], 1) * (w_i != 0)[:, None])
            if case["kind"] != "loss":
                d = torch.exp(z / T - lse)
                d.scatter_add_(1, index.clamp(min=0), -p)
                parts[2].append(d * (T * w_i)[:, None])
        loss, stats, grad = (torch.cat(x) if x else None for x in parts)
        return {"loss": (loss, stats), "step": (loss, stats, grad), "grad": grad}[case["kind"]]
    k, m, n = case["k"], case["m"], case["n"]
    signs = torch.tensor([0.0, 1.0, math.nan, -1.0], dtype=torch.float64, device="cuda")

    def dense(words, length):
        out = torch.empty((k, words.shape[1], 16), dtype=torch.float64, device="cuda")
        for e in range(16):
            out[:, :, e] = signs[((words >> (2 * e)) & 3).long()]
        return out.view(k, -1)[:, :length].contiguous()

    B, C = dense(s["B"], m), dense(s["C"], n)
    back = torch.mm(s["dY"].double(), B.t().contiguous())
    dD = (back * torch.mm(s["X"].double(), C.t().contiguous())).sum(0)
    return torch.mm(back * s["D"].double(), C), dD
