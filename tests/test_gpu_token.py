"""Cross entropy through an output matrix and its gradient against their definitions in 64 bits.

Tolerances, from the arithmetic alone.  A logit is a sum of n products in fp32: off by at most
ez = n 2^-23 max_v sum_j |x_j w_vj| (one rounding of 2^-24 a product and a sum, twice that for sums that
truncate).  exp(d) is off by 2^-24 |d| log2 e + 2^-23 of itself and d exp(d) <= 0.37, so a sum of exponentials
and a probability by the relative e = 2 ez + 2^-21.  P is rounded to the type (half an eps; for fp16 at
least 2^-39 of the largest weight, the smallest step of a number scaled to 2^14 or more); exp(d) below
2^-126 and a P below it count as 0, so P is off by up to (g + 1) 2^-126 besides.  The products of P are
fp32 sums like the logits, and the result is rounded to its type (half an eps, and half its smallest step)."""

import pytest
import torch

import expanded_rank_matrix_amd as erm

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def inputs(rows, n, vocab, dtype, seed=0, scale=2.0):
    g = torch.Generator().manual_seed(1000 * seed + rows + 7 * n + 13 * vocab)
    x = (torch.randn((rows, n), generator=g) * scale).to(dtype).cuda()
    w = (torch.randn((vocab, n), generator=g) * n**-0.5).to(dtype).cuda()
    target = torch.randint(0, vocab, (rows,), generator=g).cuda()
    weight = (torch.rand((rows,), generator=g) + 0.1).cuda()
    return x, w, target, weight


def definition(x, w, target, weight):
    """The outputs in 64 bits and how far they may be off: (loss, stats, dX, dW), (the same)."""
    dt = x.dtype
    half, f = (0.0 if dt == torch.float32 else torch.finfo(dt).eps / 2), torch.finfo(dt)
    rows, n = x.shape
    vocab = w.shape[0]
    kept = (target >= 0) & (target < vocab) & (weight != 0)
    X, W, g = x.double(), w.double(), weight.double()
    X = torch.where(kept[:, None], X, 0.0)
    at = torch.where(kept, target, 0).long()[:, None]
    z = X @ W.t().contiguous()
    lse = torch.logsumexp(z, 1)
    top = z.amax(1)
    loss = (lse - z.gather(1, at)[:, 0]) * g
    S = torch.exp(lse - top)
    P = torch.exp(z - lse[:, None])
    P = P.scatter_add(1, at, torch.full_like(at, -1, dtype=torch.float64)) * g[:, None]
    zero = torch.zeros((), dtype=torch.float64, device=x.device)
    loss, P = torch.where(kept, loss, zero), torch.where(kept[:, None], P, zero)
    stats = torch.where(kept[:, None], torch.stack([top, S], 1), zero)
    Wt, Xt = W.abs().t().contiguous(), X.abs()
    ez = n * 2.0**-23 * (Xt @ Wt).amax(1)
    e = 2 * ez + 2.0**-21
    G = torch.where(kept, g.abs(), zero)
    least = float(G.max()) * 2.0**-39 if dt == torch.float16 else 0.0
    dP = P.abs() * (half + e[:, None]) + least + (G[:, None] + 1) * 2.0**-126
    dP.scatter_add_(1, at, (G * (2.0**-22 + e) * (1 + half))[:, None])  # a difference of numbers up to g
    dP = torch.where(kept[:, None], dP, zero)
    dX, dW = P @ W, P.t().contiguous() @ X
    small = f.smallest_normal * f.eps / 2
    out = lambda v, d, k, m: d * (1 + half + 2.0**-24) + v.abs() * (half + 2.0**-23) + k * 2.0**-23 * m + small  # noqa: E731
    tx = out(dX, dP @ W.abs(), vocab, P.abs() @ W.abs())
    tw = out(dW, dP.t().contiguous() @ Xt, rows, P.abs().t().contiguous() @ Xt)
    tl = G * (2 * ez + 2.0**-21) + loss.abs() * 2.0**-23
    ts = torch.stack([ez + top.abs() * 2.0**-24, S * (e + 2.0**-23)], 1)
    return (loss, stats, dX, dW), (tl, ts, tx, tw)


def near(got, want, tol, name):
    off = (got.double() - want).abs()
    assert not torch.isnan(got).any(), f"{name}: NaN"
    worst = float((off / tol.clamp(min=1e-300)).where(off > 0, torch.zeros_like(off)).max()) if off.numel() else 0.0
    assert worst <= 1.0, f"{name}: {worst:.3g} of the tolerance"


def check(x, w, target, weight, int32=False, **how):
    t = target.int() if int32 else target
    want, tol = definition(x, w, target, weight)
    got = erm.token_loss(x, w, t, weight=weight, grad=True, **how)
    for a, b, c, name in zip(got, want, tol, ("loss", "stats", "dX", "dW")):
        near(a, b, c, name)
    loss, stats = erm.token_loss(x, w, t, weight=weight)
    assert torch.equal(loss, got[0]) and torch.equal(stats, got[1])
    dX, dW = erm.token_grad(x, w, stats, t, grad_loss=weight)
    near(dX, want[2], tol[2], "dX alone")
    near(dW, want[3], tol[3], "dW alone")
    return got


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,n,vocab", [
    (1, 1, 1), (1, 8, 2), (2, 3, 5), (1, 64, 1000), (31, 64, 129), (32, 200, 128), (33, 72, 300), (64, 128, 257),
    (65, 77, 511), (100, 256, 512), (128, 129, 700), (129, 64, 256), (200, 300, 1021), (256, 520, 255), (257, 48, 1300),
    (300, 1000, 700), (600, 136, 2051)])
def test_matches_definition(rows, n, vocab, dtype):
    check(*inputs(rows, n, vocab, TYPES[dtype]), int32=rows % 2 == 0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [64, 61])
def test_several_pieces_of_the_vocabulary(n, dtype):
    """4096 rows of 16 bits: pieces of 16384 words (8192 of fp32)."""
    x, w, target, weight = inputs(4000, n, 20011, TYPES[dtype])
    target[::3] = 16384 + torch.arange(len(target[::3]), device="cuda") % 3627
    check(x, w, target, weight)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [20, 300])
def test_rows_that_do_not_count_are_not_read(rows, dtype):
    x, w, target, weight = inputs(rows, 72, 333, TYPES[dtype], 1)
    clean = x.clone()
    bad = torch.arange(rows, device="cuda") % 3 == 1
    target[bad] = torch.tensor([-100, 333, -1, 2**31 - 1], device="cuda")[torch.arange(int(bad.sum())) % 4]
    other = torch.arange(rows, device="cuda") % 7 == 0
    weight[other] = 0.0
    x[bad | other] = float("nan")
    clean[bad | other] = 0
    want, tol = definition(clean, w, target, weight)
    for a, b, c, name in zip(erm.token_loss(x, w, target, weight=weight, grad=True), want, tol, ("loss", "stats", "dX", "dW")):
        near(a, b, c, name)
        if name != "dW":
            assert not a[bad | other].any()


@pytest.mark.parametrize("rows", [0, 1, 40, 300])
def test_no_row_counts(rows):
    x, w, target, weight = inputs(rows, 40, 100, torch.bfloat16)
    target[:] = -100
    loss, stats, dX, dW = erm.token_loss(x, w, target, weight=weight, grad=True)
    assert loss.shape == (rows,) and dX.shape == x.shape and dW.shape == w.shape
    for t in (loss, stats, dX, dW):
        assert not t.any()
    dX, dW = erm.token_grad(x, w, stats, target)
    assert not dX.any() and not dW.any()


@pytest.mark.parametrize("dtype", TYPES)
def test_strided_rows_and_outputs_beside_other_data(dtype):
    dt = TYPES[dtype]
    x, w, target, weight = inputs(70, 41, 300, dt)
    xs, ws = torch.zeros((70, 60), dtype=dt, device="cuda"), torch.zeros((300, 53), dtype=dt, device="cuda")
    xs[:, 3:44], ws[:, 1:42] = x, w
    rx, rw = torch.full((70, 50), 7.0, dtype=dt, device="cuda"), torch.full((301, 45), 7.0, dtype=dt, device="cuda")
    got = check(x, w, target, weight)
    out = erm.token_loss(xs[:, 3:44], ws[:, 1:42], target, weight=weight, out=(rx[:, 2:43], rw[:300, 3:44]))
    for a, b in zip(out, got):
        assert torch.equal(a, b)
    for room, c in ((rx, 2), (rw, 3)):
        assert (room[:, :c] == 7).all() and (room[:, c + 41:] == 7).all()
    assert (rw[300] == 7).all()


def test_gradient_in_the_place_of_the_rows():
    x, w, target, weight = inputs(90, 64, 500, torch.bfloat16)
    want = erm.token_loss(x, w, target, weight=weight, grad=True, need_dW=False)
    got = erm.token_loss(x, w, target, weight=weight, need_dW=False, out=(x, None))
    assert got[2].data_ptr() == x.data_ptr() and torch.equal(x, want[2]) and got[3] is None and want[3] is None


@pytest.mark.parametrize("which", [(True, False), (False, True)])
def test_one_gradient_alone(which):
    x, w, target, weight = inputs(140, 96, 800, torch.float16)
    _, stats, *both = erm.token_loss(x, w, target, weight=weight, grad=True)
    one = erm.token_grad(x, w, stats, target, grad_loss=weight, need_dX=which[0], need_dW=which[1])
    for a, b, need in zip(one, both, which):
        assert (a is None) == (not need)
        if need:
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_small_weights_keep_their_gradient(dtype):
    """A mean over many tokens: g of 2^-20, far below fp16's smallest numbers once times a probability."""
    x, w, target, weight = inputs(50, 64, 4000, TYPES[dtype])
    _, stats = erm.token_loss(x, w, target)
    want, _ = definition(x, w, target, torch.ones_like(weight))
    g = torch.full_like(weight, 2.0**-20 if dtype == "bf16" else 2.0**-8)
    dX, dW = erm.token_grad(x, w, stats, target, grad_loss=g)
    for got, ref in ((dX, want[2]), (dW, want[3])):
        assert float((got.double() - ref * float(g[0])).norm() / (ref * float(g[0])).norm()) < 0.01


def test_large_logits_and_sure_rows():
    x, w, target, weight = inputs(64, 32, 300, torch.float32, scale=60.0)
    check(x, w, target, weight)
    top = (x.double() @ w.double().t()).argmax(1)
    check(x, w, top, weight)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_bad_values_show(value):
    x, w, target, weight = inputs(40, 64, 300, torch.bfloat16)
    x[7, 3] = value
    loss, stats, dX, dW = erm.token_loss(x, w, target, weight=weight, grad=True)
    assert torch.isnan(loss[7]) and torch.isnan(dX[7]).all() and torch.isnan(dW).all()
    rest = torch.arange(40, device="cuda") != 7
    assert not torch.isnan(loss[rest]).any() and not torch.isnan(dX[rest]).any()
    x, w, target, weight = inputs(40, 64, 300, torch.bfloat16)
    w[250, 1] = float("nan")
    loss, stats, dX, dW = erm.token_loss(x, w, target, weight=weight, grad=True)
    assert torch.isnan(loss).all() and torch.isnan(dX).all() and torch.isnan(dW).all()


def test_gradient_against_differences():
    """fp32; the loss's sum along a direction, by central differences of the fp64 definition and of the kernel."""
    x, w, target, weight = inputs(37, 24, 90, torch.float32)
    _, _, dX, dW = erm.token_loss(x, w, target, weight=weight, grad=True)
    for k, (v, d) in enumerate(((x, dX), (w, dW))):
        u = torch.randn(v.shape, generator=torch.Generator().manual_seed(k)).cuda()
        h = 2.0**-6
        at = lambda s: [(v + s * u) if a is v else a for a in (x, w)]  # noqa: E731
        up, down = (float(definition(*at(s), target, weight)[0][0].sum()) for s in (h, -h))
        slope = float((d.double() * u.double()).sum())
        # the third derivative's share of a central difference, h^2 / 6 times at most sum |g| (2 max |u . z'|)^3
        z = (u.double() @ w.double().t() if k == 0 else x.double() @ u.double().t()).abs().max()
        bound = float(weight.sum()) * (2 * float(z)) ** 3 * h * h / 6 + 1e-3
        assert abs((up - down) / (2 * h) - slope) < bound
        lo, hi = (erm.token_loss(*at(s), target, weight=weight)[0].double().sum() for s in (-h, h))
        assert abs(float(hi - lo) / (2 * h) - slope) < bound


def test_runs_are_identical_and_streams_independent():
    a, b = inputs(300, 128, 3000, torch.bfloat16), inputs(77, 200, 900, torch.float16)
    want = [erm.token_loss(*s[:3], weight=s[3], grad=True) for s in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = [erm.token_loss(*s[:3], weight=s[3], grad=True, stream=st) for s, st in zip((a, b), streams)]
        torch.cuda.synchronize()
        for g, r in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(g, r))


def test_captured_and_replayed():
    x, w, target, weight = inputs(200, 96, 1500, torch.bfloat16)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        erm.token_loss(x, w, target, weight=weight, grad=True)
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        r1 = erm.token_loss(x, w, target, weight=weight, grad=True)
    with torch.cuda.graph(g2):
        r2 = erm.token_grad(x, w, r1[1], target, grad_loss=weight)
    for seed in range(4):
        nx, nw, nt, ng = inputs(200, 96, 1500, torch.bfloat16, seed + 5)
        nt[seed::5] = -100
        for t, v in ((x, nx), (w, nw), (target, nt), (weight, ng)):
            t.copy_(v)
        g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        want = erm.token_loss(nx, nw, nt, weight=ng, grad=True)
        assert all(torch.equal(p, q) for p, q in zip(r1, want))
        want = erm.token_grad(nx, nw, want[1], nt, grad_loss=ng)
        assert all(torch.equal(p, q) for p, q in zip(r2, want))


def test_offsets_past_32_bits():
    """W's rows 2^17 elements apart: the last lies 2^32 bytes and more behind the first."""
    n, vocab, ld = 32, 18000, 1 << 17
    room = torch.empty(vocab * ld, dtype=torch.bfloat16, device="cuda")
    w = room.as_strided((vocab, n), (ld, 1))
    x, v, target, weight = inputs(40, n, vocab, torch.bfloat16)
    w.copy_(v)
    target[::2] = vocab - 1 - torch.arange(20, device="cuda")
    got = erm.token_loss(x, w, target, weight=weight, grad=True)
    want = erm.token_loss(x, v, target, weight=weight, grad=True)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_binding_refusals():
    x, w, target, weight = inputs(6, 16, 20, torch.bfloat16)
    ok = lambda **k: erm.token_loss(**{**dict(X=x, W=w, target=target, weight=weight), **k})  # noqa: E731
    for bad in (dict(X=x.cpu()), dict(W=w.float()), dict(W=w[:, :8]), dict(target=target[:5]), dict(target=target.float()),
                dict(weight=weight[:5]), dict(weight=weight.double()), dict(X=x.t()), dict(X=x[:1].expand(6, 16)),
                dict(out=(x[:5], None)), dict(out=(None, w.float())), dict(W=None), dict(target=None)):
        with pytest.raises(ValueError):
            ok(**bad)
    with pytest.raises(ValueError):
        erm.token_grad(x, w, None, target)
    with pytest.raises(ValueError):
        erm.token_grad(x, w, torch.zeros(6, 2, device="cuda"), target, need_dX=False, need_dW=False)
    with pytest.raises(erm.ExterndError):
        ok(out=(torch.empty_like(x), w))
    with pytest.raises(erm.ExterndError):
        ok(out=(w[:6], torch.empty_like(w)))
