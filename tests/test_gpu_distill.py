"""The distillation loss and its gradient against their definitions in 64 bits.

Tolerances, from the kernel's arithmetic.  x = (z - m) / T is formed by one fp32 subtraction and one
product with a rounded constant (3 relative roundings, eps = 2^-24 each), exp2 is good to one unit in
the last place (2 eps), a thread adds at most V / 256 + 8 terms in fp32 and rescales its sum at each
new maximum (counted as 2 eps each, at most V / 2048 + 1 of them):
  rel(S) <= 2 eps + 3 eps E|x| + eps (V / 256 + 8) + 2 eps (V / 2048 + 1),   E|x| <= log V
  p: expf (4 eps) over a sum of the same, x in fp64: 8 eps;  q: 3 eps |x| + 4 eps + rel(S)
  loss: w T^2 (rel(S) + 16 eps max |log p - log q|) + 2 eps |loss|
  dz:   w T (q (rel q + 2 eps) + 10 eps p + 2^-126) + half a step of its type
The 2^-126: the hardware's exp2 returns 0 where its result is below the smallest normal number, so an
element with exp(x) < 2^-126 has q = 0 instead of exp(x) / S <= 2^-126 (S >= 1, the largest logit's
own term), which w T multiplies."""

import numpy as np
import pytest
import torch

import expanded_rank_matrix_amd as erm

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 2.0**-24


def make(rows, vocab, top, dtype, seed, spread=3.0):
    """Student logits, teacher logits and their indices; the entries of a row are distinct."""
    g = torch.Generator().manual_seed(seed)
    z = (torch.randn((rows, vocab), generator=g) * spread).to(dtype)
    t = z.float() + torch.randn((rows, vocab), generator=g)
    a, i = torch.topk(t, min(top, vocab), dim=1)
    if top > vocab:
        pad = top - vocab
        a = torch.cat([a, torch.zeros((rows, pad))], 1)
        i = torch.cat([i, torch.full((rows, pad), -1)], 1)
    return z, a.contiguous(), i.to(torch.int32).contiguous()


def reference(z, a, i, T, w):
    """(loss, max, S, dz, terms): the definition in 64 bits on the CPU, duplicates and all."""
    z, a, i = z.cpu().double(), a.cpu().double(), i.cpu().long()
    rows, V = z.shape
    w = torch.ones(rows, dtype=torch.float64) if w is None else w.cpu().double()
    m = z.amax(1)
    x = (z - m[:, None]) / T
    S = x.exp().sum(1)
    q = x.exp() / S[:, None]
    valid = (i >= 0) & (i < V) & (a > -np.inf)
    at = torch.where(valid, i, 0)
    some = valid.any(1)
    p = torch.softmax(torch.where(valid, a, -np.inf) / T, 1)
    p = torch.where(valid & some[:, None], p, 0.0)
    logq = x.gather(1, at) - S.log()[:, None]
    d = torch.where(p > 0, p.log() - logq, 0.0)
    loss = w * T * T * (p * d).sum(1)
    ps = torch.zeros_like(q).scatter_add_(1, at, p)
    dz = (w * T)[:, None] * (q * some[:, None] - ps)
    return loss, m, S, dz, (w, x, q, ps, d.abs().amax(1))


def check(out, z, a, i, T=1.0, w=None, grad_only=None):
    want, m, S, dz, (wt, x, q, ps, far) = reference(z, a, i, T, w)
    V = z.shape[1]
    relS = EPS * (2 + 3 * np.log(V) + V / 256 + 8 + 2 * (V / 2048 + 1))
    kept = wt != 0
    if grad_only is None:
        loss, stats = out[0].cpu().double(), out[1].cpu().double()
        assert torch.equal(stats[:, 0], torch.where(kept, m, 0.0))
        assert ((stats[:, 1] - S * kept).abs() <= (relS + EPS) * S).all()
        tol = wt.abs() * T * T * (relS + 16 * EPS * far) + 2 * EPS * want.abs()
        off = (loss - want).abs()
        assert (off <= tol).all(), f"loss off by {float((off / tol.clamp(min=1e-300)).max()):.3g} of the tolerance"
    d = out[2] if grad_only is None and len(out) == 3 else grad_only
    if d is not None:
        f = torch.finfo(d.dtype)
        half = f.eps / 2
        tol = (wt.abs() * T)[:, None] * (q * (relS + EPS * (3 * torch.where(q > 0, x.abs(), 0.0) + 8)) + 10 * EPS * ps + 2.0**-126)
        tol = tol * (1 + half) + dz.abs() * half + f.smallest_normal * half
        off = (d.cpu().double() - dz).abs()
        assert (off <= tol).all(), f"gradient off by {float((off / tol).max()):.3g} of the tolerance"


def run(z, a, i, T=1.0, w=None, grad=True):
    w = None if w is None else w.cuda()
    z, a, i = z.cuda(), a.cuda(), i.cuda()
    out = erm.distill_loss(z, a, i, T, w, grad=grad)
    check(out, z, a, i, T, w)
    d = erm.distill_grad(z, out[1], a, i, T, w)
    check(None, z, a, i, T, w, grad_only=d)
    return out


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab,top", [(1, 1, 1), (3, 7, 3), (2, 8, 8), (5, 9, 20), (4, 255, 16), (1100, 100, 7),
                                            (3, 2048, 64), (2, 2049, 1), (6, 8192, 128), (3, 40001, 256), (1, 131072, 64),
                                            (1030, 4099, 33), (2, 70000, 1024), (1025, 8201, 9), (1024, 16385, 5),
                                            (1024, 32769, 70), (1024, 65543, 3)])
def test_loss_and_gradient(rows, vocab, top, dtype):
    z, a, i = make(rows, vocab, top, TYPES[dtype], rows + vocab + top)
    run(z, a, i)


@pytest.mark.parametrize("T", [0.25, 2.0, 7.5])
def test_temperatures_weights_and_types(T):
    z, a, i = make(37, 5000, 40, torch.bfloat16, 3)
    w = torch.rand(37, generator=torch.Generator().manual_seed(1)) * 3 - 1
    w[::5] = 0
    for at in TYPES.values():
        for it in (torch.int32, torch.int64):
            run(z, a.to(at), i.to(it), T, w)


def test_weight_zero_rows_are_not_read():
    z, a, i = make(40, 9000, 16, torch.float32, 9)
    w = torch.ones(40)
    w[3], w[17] = 0, 0
    z[3], a[17], z[17, 5] = float("nan"), float("nan"), float("inf")
    zc, ac, ic, wc = z.cuda(), a.cuda(), i.cuda(), w.cuda()
    loss, stats, d = erm.distill_loss(zc, ac, ic, weight=wc, grad=True)
    d2 = erm.distill_grad(zc, stats, ac, ic, grad_loss=wc)
    for t in (loss, stats, d, d2):
        assert not t[[3, 17]].any() and torch.isfinite(t).all()
    keep = [r for r in range(40) if r not in (3, 17)]
    check((loss[keep], stats[keep], d[keep]), z[keep], a[keep], i[keep])


@pytest.mark.parametrize("rows,vocab", [(30, 600), (2, 20000), (1100, 300)])
def test_short_lists_duplicates_and_bad_indices(rows, vocab):
    z, a, i = make(rows, vocab, 48, torch.float32, 21)
    i[:, 40:] = -1
    i[0, :] = -1                                  # no entry at all
    i[1, 5], i[1, 6], i[1, 7] = vocab, 2**31 - 1, -(2**31)
    if rows > 3:
        i[2, :40] = i[2, 0]                       # one index 40 times
        i[3, 1::2] = i[3, 0::2]                   # each twice
        a[4, 3:9] = -float("inf")
    out = run(z, a, i, 2.0)
    assert out[0][0] == 0 and not out[2][0].any()
    a[0] = -float("inf")
    i[0] = 1
    out = run(z, a, i, 2.0)                       # entries, but none with a logit
    assert out[0][0] == 0 and not out[2][0].any()


@pytest.mark.parametrize("rows,vocab", [(8, 700), (8, 30000)])
def test_masked_logits(rows, vocab):
    """Logits of -inf and of the type's lowest value off the teacher's entries: q is 0 there."""
    for dtype in TYPES.values():
        z, a, i = make(rows, vocab, 5, dtype, 13)
        lowest = torch.finfo(dtype).min
        free = torch.ones((rows, vocab), dtype=torch.bool).scatter_(1, i.long(), False)
        z[0][free[0]] = -float("inf")
        z[1][free[1]] = lowest
        z[2][free[2] & (torch.arange(vocab) % 3 == 0)] = -float("inf")
        z[3, :] = lowest                          # a uniform row
        out = run(z, a, i)
        assert not out[2][0].cpu()[free[0]].any()
        if dtype == torch.float32 or dtype == torch.bfloat16:
            assert not out[2][1].cpu()[free[1]].any()


@pytest.mark.parametrize("rows,vocab", [(12, 900), (12, 30000), (1100, 500)])
def test_nan_and_infinity_stay_in_their_rows(rows, vocab):
    z, a, i = make(rows, vocab, 9, torch.float32, 31)
    zb, ab = z.clone(), a.clone()
    zb[0, 7] = float("nan")
    zb[1, 7] = float("inf")
    zb[2, :] = -float("inf")
    ab[3, 2] = float("nan")
    ab[4, 2] = float("inf")
    zb[5, i[5, 0]] = -float("inf")                # the student gives a wanted token nothing
    loss, stats, d = erm.distill_loss(zb.cuda(), ab.cuda(), i.cuda(), grad=True)
    d2 = erm.distill_grad(zb.cuda(), stats, ab.cuda(), i.cuda())
    assert torch.isnan(loss[:5]).all() and loss[5] == float("inf")
    for g in (d, d2):
        assert torch.isnan(g[:3]).all() and torch.isnan(g[3:5]).any(1).all()
        assert torch.isfinite(g[5:]).all()
    rest = erm.distill_loss(z[6:].cuda(), a[6:].cuda(), i[6:].cuda(), grad=True)
    if rows < 100:  # the same split of the rows
        check((loss[6:], stats[6:], d[6:]), z[6:], a[6:], i[6:])
    else:
        assert torch.equal(loss[6:], rest[0]) and torch.equal(d[6:], rest[2])


def test_strided_rows_and_gradient_in_place():
    for rows in (3, 1100):
        z, a, i = make(rows, 5001, 12, torch.bfloat16, 8)
        room = torch.zeros((rows, 5100), dtype=torch.bfloat16, device="cuda")
        room[:, 7:5008] = z.cuda()
        view = room[:, 7:5008]
        plain = erm.distill_loss(z.cuda(), a.cuda(), i.cuda(), grad=True)
        out = torch.full((rows, 5003), 9.0, dtype=torch.bfloat16, device="cuda")
        got = erm.distill_loss(view, a.cuda(), i.cuda(), out=out[:, 1:5002])
        assert got[2].data_ptr() == out[:, 1:5002].data_ptr()
        for x, y in zip(got, plain):
            assert torch.equal(x, y)
        assert (out[:, 0] == 9).all() and (out[:, 5002:] == 9).all()
        twin = room.clone()
        loss, stats = erm.distill_loss(view, a.cuda(), i.cuda())
        assert torch.equal(loss, plain[0]) and torch.equal(stats, plain[1])
        want = erm.distill_grad(view, stats, a.cuda(), i.cuda())
        erm.distill_grad(view, stats, a.cuda(), i.cuda(), out=view)
        assert torch.equal(view, want)
        view = twin[:, 7:5008]
        got = erm.distill_loss(view, a.cuda(), i.cuda(), out=view)
        for x, y in zip(got, plain):
            assert torch.equal(x, y)
        assert not twin[:, :7].any() and not twin[:, 5008:].any()


def test_gradient_against_differences():
    z, a, i = make(4, 300, 10, torch.float32, 5, spread=1.0)
    T = 1.5
    d = erm.distill_loss(z.cuda(), a.cuda(), i.cuda(), T, grad=True)[2].cpu().double()
    g = torch.Generator().manual_seed(2)
    h = 1e-5
    for _ in range(5):
        v = torch.randn((4, 300), generator=g, dtype=torch.float64)
        up, down = (reference(z.double() + s * h * v, a, i, T, None)[0] for s in (1, -1))
        # fourth-order terms and fp64 cancellation stay below 1e-7 at this step; dz's own 2^-20
        assert torch.allclose((up - down) / (2 * h), (d * v).sum(1), rtol=1e-5, atol=1e-5)


def test_deterministic_streams_and_graph():
    sets = [[t.cuda() for t in make(r, v, 20, torch.float32, r)] for r, v in ((5, 30000), (1050, 400))]
    want = [erm.distill_loss(*s, 2.0, grad=True) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [erm.distill_loss(*s, 2.0, grad=True, stream=st) for _ in range(3) for s, st in zip(sets, streams)]
    torch.cuda.synchronize()
    for k, o in enumerate(got):
        for x, y in zip(o, want[k % 2]):
            assert torch.equal(x, y)
    z, a, i = sets[0]
    static = z.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = erm.distill_loss(static, a, i, 2.0, grad=True)
        d = erm.distill_grad(static, out[1], a, i, 2.0)
    for k in range(4):
        static.copy_(z * (1 + k))
        graph.replay()
        torch.cuda.synchronize()
        eager = erm.distill_loss(static, a, i, 2.0, grad=True)
        for x, y in zip(out, eager):
            assert torch.equal(x, y), k
        assert torch.equal(d, erm.distill_grad(static, eager[1], a, i, 2.0)), k


def test_offsets_past_32_bits():
    """70 000 x 32 768 fp16 logits: element offsets pass 2^31."""
    rows, vocab = 70000, 32768
    z, a, i = make(64, vocab, 8, torch.float16, 4)
    big = z.cuda().repeat((rows + 63) // 64, 1)[:rows]
    pick = torch.arange(rows, device="cuda") % 64
    out = erm.distill_loss(big, a.cuda()[pick].contiguous(), i.cuda()[pick].contiguous(), out=big)
    few = erm.distill_loss(z.repeat(32, 1).cuda(), a.repeat(32, 1).cuda(), i.repeat(32, 1).cuda(), grad=True)
    for x, y in zip(out, few):  # 2048 rows take whole-row workgroups, as 70 000 do
        assert torch.equal(x[:64], y[:64]) and torch.equal(x[69952:], y[: rows - 69952])


def test_empty_and_binding_refusals():
    z, a, i = (t.cuda() for t in make(3, 50, 4, torch.float32, 1))
    loss, stats, d = erm.distill_loss(z[:0], a[:0], i[:0], grad=True)
    assert loss.shape == (0,) and stats.shape == (0, 2) and d.shape == (0, 50)
    assert erm.distill_grad(z[:0], stats, a[:0], i[:0]).shape == (0, 50)
    stats = erm.distill_loss(z, a, i)[1]
    w = torch.ones(3, device="cuda")
    bad = [lambda: erm.distill_loss(z.double(), a, i), lambda: erm.distill_loss(z[0], a, i),
           lambda: erm.distill_loss(z, a[:2], i), lambda: erm.distill_loss(z, a, i[:, :3].contiguous()),
           lambda: erm.distill_loss(z, a, i.short()), lambda: erm.distill_loss(z, a.double(), i),
           lambda: erm.distill_loss(z, a.cpu(), i), lambda: erm.distill_loss(z, a, i, weight=w[:2]),
           lambda: erm.distill_loss(z, a, i, weight=w.double()), lambda: erm.distill_loss(z, a, i, out=z[:, :49]),
           lambda: erm.distill_loss(z, a, i, out=z.half()), lambda: erm.distill_loss(z.t().contiguous().t(), a, i),
           lambda: erm.distill_loss(z, a.t().contiguous().t(), i), lambda: erm.distill_loss(z[:1].expand(3, 50), a, i),
           lambda: erm.distill_grad(z, stats[:2], a, i), lambda: erm.distill_grad(z, stats.double(), a, i),
           lambda: erm.distill_grad(z, stats, a, i, grad_loss=w[:1])]
    for k, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {k} was not refused")
    for T in (0.0, float("nan"), 1e4):
        with pytest.raises(erm.ExterndError):
            erm.distill_loss(z, a, i, T)


@pytest.mark.parametrize("rows,vocab", [(3, 400), (2, 9000), (1030, 400), (1030, 8205)])
def test_small_teacher_probabilities_keep_their_bits(rows, vocab):
    """Teacher entries down to p = e^-80 whose students' logits are far below: the gradient there is
    -w T p, good to 10 eps of p however small it is, for single indices and for repeated ones."""
    g = torch.Generator().manual_seed(rows + vocab)
    top, T = 40, float(np.float32(0.7))  # as the entry takes it: 0.7 in 64 bits is 80 1.7e-8 away in an exponent
    z = torch.randn((16, vocab), generator=g)
    a = -56.0 * torch.rand((16, top), generator=g)
    a[:, 0] = 0.0
    i = torch.stack([torch.randperm(vocab, generator=g)[:top] for _ in range(16)])
    i[:, 30:] = i[:, 20:30]                        # ten indices twice, their p far apart
    i[:, 38:] = i[:, 21:23]                        # two of them three times
    z.scatter_(1, i, -150.0)
    z, a, i = (t.repeat((rows + 15) // 16, 1)[:rows].contiguous() for t in (z, a, i.to(torch.int32)))
    w = torch.full((rows,), 2.0**30)
    zc, ac, ic, wc = z.cuda(), a.cuda(), i.cuda(), w.cuda()
    out = erm.distill_loss(zc, ac, ic, T, wc, grad=True)
    d = erm.distill_grad(zc, out[1], ac, ic, T, wc)
    few = min(rows, 16)
    check([t[:few] for t in out], z[:few], a[:few], i[:few], T, w[:few])
    check(None, z[:few], a[:few], i[:few], T, w[:few], grad_only=d[:few])
    for t in (*out, d):
        assert torch.equal(t, t[:few].repeat((rows + 15) // 16, *[1] * (t.dim() - 1))[:rows])


def furthest_temperature():
    """A temperature whose log2 e / T lies nearly half a step from the nearest fp32 number."""
    t = np.float32(1.4426) + np.arange(300, dtype=np.float32) * np.float32(2.0**-23)
    c = np.log2(np.e) / t.astype(np.float64)
    return float(t[np.argmax(np.abs(c.astype(np.float32).astype(np.float64) / c - 1))])


@pytest.mark.parametrize("rows,vocab", [(4, 300), (3, 9000), (1030, 300), (1030, 8205), (1026, 33001)])
def test_exponents_lose_only_their_rounding(rows, vocab):
    """Logits whose differences from the row's largest are exact, one of them far above the others, so
    S = 1 + vocab e^-30 (its error is below eps).  The exponent y = (z - m) log2(e) / T then rounds once,
    by 2^-24 |y|, which is 2^-24 |x| in its power.  Besides: exp2 2 eps, 1 / S, its product with w T, the
    product with it and S's own rounding eps each, second orders: 8 eps.  A constant rounded to fp32 would
    add up to eps |x|."""
    T = furthest_temperature()
    g = torch.Generator().manual_seed(rows + vocab)
    base = -torch.randint(int(30 * 8 * 1.45), int(84 * 8 * 1.44), (16, vocab), generator=g).float() / 8
    base[:, 5] = 0
    z = base.repeat((rows + 15) // 16, 1)[:rows].contiguous()
    w = 2.0**40
    a, i = torch.zeros((rows, 1)), torch.full((rows, 1), 5, dtype=torch.int32)
    zc, ac, ic, wc = z.cuda(), a.cuda(), i.cuda(), torch.full((rows,), w).cuda()
    _, stats, d = erm.distill_loss(zc, ac, ic, T, wc, grad=True)
    x = base[:rows].double() / T
    q = x.exp() / x.exp().sum(1, keepdim=True)
    tol = w * T * q * EPS * (x.abs() + 8)
    for got in (d, erm.distill_grad(zc, stats, ac, ic, T, wc)):
        off = (got[:16].cpu().double() - w * T * q).abs()
        off[:, 5], tol[:, 5] = 0, 1
        assert (off <= tol).all(), float((off / tol).max())
        assert torch.equal(got, got[:16].repeat((rows + 15) // 16, 1)[:rows])


def test_missing_tensors_are_refused():
    z, a, i = (t.cuda() for t in make(3, 50, 4, torch.float32, 1))
    stats = torch.zeros((3, 2), device="cuda")
    for call in (lambda: erm.distill_loss(None, a, i), lambda: erm.distill_loss(z, None, i),
                 lambda: erm.distill_loss(z, a, None), lambda: erm.distill_grad(z, None, a, i),
                 lambda: erm.distill_grad(None, stats, a, i), lambda: erm.distill_grad(z, stats, None, i),
                 lambda: erm.distill_grad(z, stats, a, None)):
        with pytest.raises(ValueError):
            call()


def test_gradient_beside_the_logits_and_over_them():
    """Both as columns of one matrix, and a single row; a shifted overlap is refused."""
    for rows in (1, 3, 1100):
        z, a, i = make(rows, 301, 12, torch.bfloat16, 8)
        room = torch.zeros((rows, 602), dtype=torch.bfloat16, device="cuda")
        room[:, :301] = z.cuda()
        want = erm.distill_loss(z.cuda(), a.cuda(), i.cuda(), grad=True)
        for x, y in zip(erm.distill_loss(room[:, :301], a.cuda(), i.cuda(), out=room[:, 301:]), want):
            assert torch.equal(x, y)
        assert torch.equal(room[:, :301], z.cuda())
        with pytest.raises(erm.ExterndError):
            erm.distill_loss(room[:, :301], a.cuda(), i.cuda(), out=room[:, 300:601])
        erm.distill_grad(room[:, 301:], want[1], a.cuda(), i.cuda(), out=room[:, :301])
        with pytest.raises(erm.ExterndError):
            erm.distill_grad(room[:, 301:], want[1], a.cuda(), i.cuda(), out=room[:, 1:302])


# rows held in registers between the passes: at least 1024 rows and a gradient, each number of threads and chunks
HELD = [("f32", 8205), ("f16", 16389), ("bf16", 33001), ("f32", 33001), ("f16", 66003)]


def spread(rows, vocab, top, dtype, seed):
    """`rows` rows that repeat 24 different ones."""
    z, a, i = make(24, vocab, top, dtype, seed)
    return z, a, i, torch.arange(rows) % 24


@pytest.mark.parametrize("dtype,vocab", HELD)
def test_held_rows_with_masks_weights_and_bad_lists(dtype, vocab):
    rows, T = 1030, 1.5
    z, a, i, pick = spread(rows, vocab, 40, TYPES[dtype], vocab)
    last = torch.arange(vocab) >= vocab - vocab % 8
    i[0] = -1                                                # no entry
    a[1] = -float("inf")                                     # entries, none with a logit
    i[2, 3], i[2, 4], i[2, 5] = vocab, 2**31 - 1, -(2**31)
    i[3] = i[3, 0]                                           # one index 40 times
    i[4, 1::2] = i[4, 0::2]                                  # each twice
    free = torch.ones((24, vocab), dtype=torch.bool).scatter_(1, i.clamp(0, vocab - 1).long(), False)
    z[5][free[5]] = -float("inf")
    z[6][free[6]] = torch.finfo(TYPES[dtype]).min
    z[7, :] = torch.finfo(TYPES[dtype]).min
    z[8][free[8] & last] = -float("inf")                     # the row's end masked, and all but it
    z[9][free[9] & ~last] = -float("inf")
    a[10, 3:9] = -float("inf")
    w = torch.rand(24, generator=torch.Generator().manual_seed(1)) * 3 - 1
    w[11] = 0
    z[11, 5] = float("nan")                                  # not read
    good = [r for r in range(24) if r != 11]
    zc, ac, ic, wc = (t[pick].contiguous().cuda() for t in (z, a, i, w))
    out = erm.distill_loss(zc, ac, ic, T, wc, grad=True)
    d = erm.distill_grad(zc, out[1], ac, ic, T, wc)
    check([t[:24][good] for t in out], z[good], a[good], i[good], T, w[good])
    check(None, z[good], a[good], i[good], T, w[good], grad_only=d[:24][good])
    for t in (*out, d):
        assert not t[11].any()
        assert torch.equal(t, t[:24][pick.cuda()])
    assert not out[2][0].any() and not out[2][1].any() and out[0][0] == 0 and not out[2][5].cpu()[free[5]].any()
    same = erm.distill_loss(zc, ac, ic, T, wc, out=zc)       # in the logits' place
    for x, y in zip(same, out):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype,vocab", HELD)
def test_held_rows_with_nan_and_infinity(dtype, vocab):
    z, a, i, pick = spread(1030, vocab, 9, TYPES[dtype], vocab + 1)
    plain = erm.distill_loss(*(t[pick].contiguous().cuda() for t in (z, a, i)), grad=True)
    z[0, 7], z[1, vocab - 1], z[2, 7], z[3, :] = float("nan"), float("nan"), float("inf"), -float("inf")
    a[4, 2], a[5, 2] = float("nan"), float("inf")
    z[6, i[6, 0]] = -float("inf")                            # the student gives a wanted token nothing
    out = erm.distill_loss(*(t[pick].contiguous().cuda() for t in (z, a, i)), grad=True)
    loss, stats, d = (t[:24] for t in out)
    assert torch.isnan(loss[:6]).all() and loss[6] == float("inf")
    assert torch.isnan(d[:4]).all() and torch.isnan(d[4:6]).any(1).all() and torch.isfinite(d[6:]).all()
    for x, y in zip(out, plain):
        assert torch.equal(x[7:24], y[7:24])
        assert torch.equal(torch.nan_to_num(x, 5.0), torch.nan_to_num(x[:24][pick.cuda()], 5.0))


@pytest.mark.parametrize("dtype", TYPES)
def test_vocabularies_past_the_held_ones(dtype):
    """Over 131072 logits of 16 bits or 65536 of fp32 the rows stream twice."""
    z, a, i, pick = spread(1025, 140003, 70, TYPES[dtype], 5)
    zc, ac, ic = (t[pick].contiguous().cuda() for t in (z, a, i))
    out = erm.distill_loss(zc, ac, ic, 1.5, grad=True)
    d = erm.distill_grad(zc, out[1], ac, ic, 1.5)
    check([t[:24] for t in out], z, a, i, 1.5)
    check(None, z, a, i, 1.5, grad_only=d[:24])
    for t in (*out, d):
        assert torch.equal(t, t[:24][pick.cuda()])


def test_more_rows_than_a_launch():
    """2^21 + 3 rows: the last three are a launch of their own."""
    rows = 2**21 + 3
    z, a, i = make(4096, 5, 2, torch.float32, 3)
    pick = torch.arange(rows) % 4093
    w = torch.rand(rows, generator=torch.Generator().manual_seed(2))
    zc, ac, ic, wc = (t.contiguous().cuda() for t in (z[pick], a[pick], i[pick], w))
    out = erm.distill_loss(zc, ac, ic, 2.0, wc, grad=True)
    d = erm.distill_grad(zc, out[1], ac, ic, 2.0, wc)
    for s in (slice(0, 50), slice(2**21 - 20, rows)):
        check([t[s] for t in out], z[pick[s]], a[pick[s]], i[pick[s]], 2.0, w[s])
        check(None, z[pick[s]], a[pick[s]], i[pick[s]], 2.0, w[s], grad_only=d[s])
    one = erm.distill_loss(zc, ac, ic, 2.0)
    assert torch.equal(one[0][:4093], one[0][4093:8186]) and torch.equal(one[1][pick[-3:]], one[1][-3:])
