"""The factored layer's gradient against its formula in 64 bits, and a compressed layer's whole run.

Tolerances, from the arithmetic: a vector's image is within ux = 2^-31 2^E of it per element (|x| < 2^E),
u, t, D u and the outputs round to fp32 once each (eps = 2^-24), dD's sum is fp64:
  |du_i| <= nnz(B_i) uy + eps |u_i|        |dt_i| <= nnz(C_i) ux + eps |t_i|
  |d dD_i| <= sum_b (|t| |du| + |u| |dt| + |du| |dt|) + eps |dD_i|
  |d dx_j| <= sum_i |C_ij| (|D_i| |du_i| + eps |D_i u_i| + us) + eps |dx_j|
A rounding to fp32 below the smallest normal number is off by up to half the smallest subnormal,
2^-150, whatever the value: each eps |v| above is eps |v| + 2^-150."""

import numpy as np
import pytest
import torch

import expanded_rank_matrix_amd as erm
from tests.test_oracle_apply import pack, random_factors

pytestmark = pytest.mark.gpu
EPS, SUB = 2.0**-24, 2.0**-150


def device(Bt, Ct, D):
    put = lambda p: torch.from_numpy(np.ascontiguousarray(p).view(np.int32)).cuda()
    return put(pack(Bt)), put(pack(Ct)), torch.from_numpy(np.ascontiguousarray(D, dtype=np.float32)).cuda()


def unit(v):
    """Half a unit of each row's image."""
    mx = np.max(np.abs(v), axis=1, initial=0.0)
    return np.ldexp(1.0, np.where(mx > 0, np.frexp(mx)[1], 0) - 31)[:, None]


def check(Bt, Ct, D, X, dY, dX, dD):
    B, C, d = Bt.astype(np.float64), Ct.astype(np.float64), D.astype(np.float64)
    x, y = X.astype(np.float64), dY.astype(np.float64)
    u, t = y @ B.T, x @ C.T
    du = np.count_nonzero(Bt, axis=1)[None] * unit(y) + EPS * np.abs(u) + SUB
    dt = np.count_nonzero(Ct, axis=1)[None] * unit(x) + EPS * np.abs(t) + SUB
    if dD is not None:
        want = (t * u).sum(0)
        tol = (np.abs(t) * du + np.abs(u) * dt + du * dt).sum(0) * (1 + 1e-9) + EPS * np.abs(want) + SUB
        off = np.abs(dD.cpu().numpy() - want)
        assert np.all(off <= tol), f"dD off by {np.max(off / tol):.3g} of the tolerance"
    if dX is not None:
        s = u * d
        want = s @ C
        us = 2 * unit(s)  # one binade of slack: the largest |s| may round up over a power of two
        tol = (np.abs(d) * du + EPS * np.abs(s) + SUB + us) @ np.abs(C) * (1 + 1e-6) + EPS * np.abs(want) + SUB
        off = np.abs(dX.cpu().numpy() - want)
        assert np.all(off <= tol), f"dX off by {np.max(off / tol):.3g} of the tolerance"


def run(k, m, n, batch, seed=0, scale=1.0):
    rng = np.random.default_rng(seed + k + m + n + batch)
    Bt, Ct, D = random_factors(rng, k, m, n)
    X = (rng.standard_normal((batch, n)) * scale).astype(np.float32)
    X[:, rng.integers(0, n)] *= 20
    dY = rng.standard_normal((batch, m)).astype(np.float32)
    Bp, Cp, Dd = device(Bt, Ct, D)
    Xc, Yc = torch.from_numpy(X).cuda(), torch.from_numpy(dY).cuda()
    dX, dD = erm.apply_factors_grad(Bp, Cp, Dd, m, n, Xc, Yc)
    assert tuple(dX.shape) == (batch, n) and tuple(dD.shape) == (k,)
    check(Bt, Ct, D, X, dY, dX, dD)
    one, none = erm.apply_factors_grad(Bp, Cp, Dd, m, n, None, Yc, need_dD=False)
    assert none is None and torch.equal(one, dX)
    none, one = erm.apply_factors_grad(Bp, Cp, Dd, m, n, Xc, Yc, need_dX=False)
    assert none is None and torch.equal(one, dD)
    return Bt, Ct, D, X, dY, dX, dD


@pytest.mark.parametrize("batch", [1, 2, 3, 15, 16, 17, 32, 33, 65, 130])
@pytest.mark.parametrize("k,m,n", [(1, 1, 1), (5, 7, 9), (16, 16, 16), (64, 17, 33), (300, 389, 103), (37, 1100, 17),
                                   (1003, 16, 2000)])
def test_gradient_matches_formula(k, m, n, batch):
    run(k, m, n, batch)


# both sides of the choice of kernels; whole and split tiles, ragged in every size
@pytest.mark.parametrize("k,m,n,batch", [(7680, 2560, 2560, 1), (7680, 2560, 2560, 16), (7680, 2560, 2560, 17),
                                         (7680, 2560, 2560, 40), (3001, 2999, 2503, 37), (1003, 777, 1025, 334),
                                         (1536, 1024, 1024, 300), (900, 640, 2100, 513), (64, 48, 50, 4096),
                                         (64, 48, 50, 4097), (37, 110, 17, 8200), (1, 1, 1, 5000), (130, 257, 300, 9000),
                                         (600, 5000, 7000, 5), (600, 5000, 7000, 90), (300, 200, 200, 700),
                                         (33, 70, 45, 2500), (1203, 777, 1025, 37), (1203, 777, 1025, 130)])
def test_gradient_larger_sizes(k, m, n, batch):
    run(k, m, n, batch)


# small batches straight from the packed codes: one or two tiles of components and of columns a workgroup,
# rows of a single word and of words that end inside a step, vectors that end inside a tile
@pytest.mark.parametrize("k,m,n,batch", [(4097, 17, 33, 9), (2049, 1, 1, 50), (2100, 50, 4000, 23), (513, 3000, 31, 61),
                                         (1000, 1, 700, 70), (4111, 515, 1031, 100), (640, 64, 8200, 130),
                                         (8200, 255, 257, 35), (515, 300, 12, 460), (257, 256, 4097, 250),
                                         (2560, 1024, 512, 16), (7680, 2560, 2560, 130)])
def test_gradient_from_packed_codes(k, m, n, batch):
    run(k, m, n, batch)


# long sums over few tiles: the widened products split them, each of the three in its turn
@pytest.mark.parametrize("k,m,n,batch", [(100, 60, 9000, 900), (100, 9000, 60, 900), (7680, 48, 48, 600)])
def test_gradient_of_split_products(k, m, n, batch):
    run(k, m, n, batch)


@pytest.mark.parametrize("batch", [5, 300, 4300])
def test_a_bad_vector_stays_alone(batch):
    Bt, Ct, D, X, dY, dX, _ = run(130, 75, 93, batch, seed=6)
    X[2, 5], dY[3, 7] = np.inf, np.nan
    got, _ = erm.apply_factors_grad(*device(Bt, Ct, D), 75, 93, torch.from_numpy(X).cuda(), torch.from_numpy(dY).cuda())
    good = torch.arange(batch, device="cuda") != 3  # dX does not depend on X
    assert torch.equal(got[good], dX[good])


@pytest.mark.parametrize("scale", [1e-38, 1e-42, 1e30])
@pytest.mark.parametrize("batch", [2, 20, 700, 4100])
def test_gradient_extreme_scales(batch, scale):
    run(50, 40, 60, batch, scale=scale)


@pytest.mark.parametrize("batch", [4, 50, 700, 4200])
def test_zero_parts(batch):
    Bt, Ct, D, X, dY, _, _ = run(40, 50, 60, batch)
    Z = np.zeros_like(Bt)
    Xc, Yc = torch.from_numpy(X).cuda(), torch.from_numpy(dY).cuda()
    dX, dD = erm.apply_factors_grad(*device(Z, Ct, D), 50, 60, Xc, Yc)
    assert not dX.any() and not dD.any()
    dX, dD = erm.apply_factors_grad(*device(Bt, Ct, np.zeros_like(D)), 50, 60, Xc, Yc)
    assert not dX.any() and dD.any()
    check(Bt, Ct, np.zeros_like(D), X, dY, dX, dD)
    dX, dD = erm.apply_factors_grad(*device(Bt, Ct, D), 50, 60, Xc, torch.zeros_like(Yc))
    assert not dX.any() and not dD.any()


def test_empty_and_single_vector():
    rng = np.random.default_rng(1)
    Bt, Ct, D = random_factors(rng, 30, 20, 25)
    f = device(Bt, Ct, D)
    dX, dD = erm.apply_factors_grad(*f, 20, 25, torch.zeros((0, 25), device="cuda"), torch.zeros((0, 20), device="cuda"))
    assert dX.shape == (0, 25) and dD.shape == (30,) and not dD.any()
    x, y = torch.randn(25, device="cuda"), torch.randn(20, device="cuda")
    one = erm.apply_factors_grad(*f, 20, 25, x, y)
    row = erm.apply_factors_grad(*f, 20, 25, x[None], y[None])
    assert one[0].shape == (25,) and torch.equal(one[0], row[0][0]) and torch.equal(one[1], row[1])


@pytest.mark.parametrize("batch", [3, 60, 4200])
def test_gradient_against_the_forward_pass(batch):
    """The layer is linear in X and in D: <dX, v> = <dY, layer(v)> and <dD, w> = <dY, layer with w>."""
    Bt, Ct, D, X, dY, dX, dD = run(200, 90, 110, batch, seed=3)
    B, C, Dd = device(Bt, Ct, D)
    rng = np.random.default_rng(8)
    v = torch.from_numpy(rng.standard_normal((batch, 110)).astype(np.float32)).cuda()
    w = torch.from_numpy(rng.standard_normal(200).astype(np.float32)).cuda()
    y = torch.from_numpy(dY).cuda().double()
    Yv = erm.apply_factors(B, C, Dd, 90, 110, v).double()
    Yw = erm.apply_factors(B, C, w, 90, 110, torch.from_numpy(X).cuda()).double()
    # every element is good to about 2^-22 of its terms' magnitudes; 2^-16 of the sums' leaves room
    for a, b in (((dX.double() * v).sum(), (y * Yv).sum()), ((dD.double() * w).sum(), (y * Yw).sum())):
        size = (dX.double() * v).abs().sum() + (y * Yv).abs().sum() + (dD.double() * w).abs().sum()
        assert abs(float(a - b)) <= 2.0**-16 * float(size)


def test_misaligned_inputs_out_streams_and_graph():
    for batch in (5, 70, 300, 4300):
        Bt, Ct, D, X, dY, dX, dD = run(130, 75, 93, batch, seed=5)
        f = device(Bt, Ct, D)
        put = lambda a: torch.cat([torch.zeros(1), torch.from_numpy(a).reshape(-1)]).cuda()[1:].reshape(a.shape)
        Xc, Yc = put(X), put(dY)
        got = erm.apply_factors_grad(*f, 75, 93, Xc, Yc)
        assert torch.equal(got[0], dX) and torch.equal(got[1], dD)
        out = (torch.empty_like(dX), torch.empty_like(dD))
        assert erm.apply_factors_grad(*f, 75, 93, Xc, Yc, out=out)[0] is out[0]
        assert torch.equal(out[0], dX) and torch.equal(out[1], dD)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        many = [erm.apply_factors_grad(*f, 75, 93, Xc, Yc, stream=s) for _ in range(3) for s in streams]
        torch.cuda.synchronize()
        for g in many:
            assert torch.equal(g[0], dX) and torch.equal(g[1], dD)
        static = Xc.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            g = erm.apply_factors_grad(*f, 75, 93, static, Yc)
        for r in range(4):
            static.copy_(Xc * (r + 1))
            graph.replay()
            torch.cuda.synchronize()
            want = erm.apply_factors_grad(*f, 75, 93, static, Yc)
            assert torch.equal(g[0], want[0]) and torch.equal(g[1], want[1]), r


@pytest.mark.parametrize("batch", [70, 1200])
def test_offsets_past_32_bits(batch):
    """k = 131 072 components of 32 768 outputs, 2^32 of them (as bytes where the batch is large).  Two
    vectors have a gradient, against those two alone (the inference kernels)."""
    k, m, n = 1 << 17, 1 << 15, 48
    g = torch.Generator(device="cuda").manual_seed(3)

    def codes(words):  # any word whose codes are 0, 1 or 3
        w = torch.randint(-(2**31), 2**31 - 1, (k, words), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
        return w | ((w >> 1) & 0x55555555)

    B, C = codes(m // 16), codes(n // 16)
    D = torch.randn(k, generator=g, device="cuda")
    X = torch.randn((batch, n), generator=g, device="cuda")
    dY = torch.zeros((batch, m), device="cuda")
    dY[:2] = torch.randn((2, m), generator=g, device="cuda")
    dX, dD = erm.apply_factors_grad(B, C, D, m, n, X, dY)
    wX, wD = erm.apply_factors_grad(B, C, D, m, n, X[:2].contiguous(), dY[:2].contiguous())
    assert not dX[2:].any()
    # both sides are within a few 2^-24 of their terms; the sums of 32768 and 131072 terms leave 2^-16
    assert (dX[:2] - wX).norm() <= 2.0**-16 * wX.norm() and (dD - wD).norm() <= 2.0**-16 * wD.norm()
    assert wX.norm() > 0 and wD[k // 2:].norm() > 0


def test_binding_refusals():
    rng = np.random.default_rng(1)
    B, C, D = device(*random_factors(rng, 30, 20, 25))
    x, y = torch.zeros((4, 25), device="cuda"), torch.zeros((4, 20), device="cuda")
    g = erm.apply_factors_grad
    bad = [lambda: g(B[:29], C, D, 20, 25, x, y), lambda: g(B, C.long(), D, 20, 25, x, y),
           lambda: g(B, C, D[None], 20, 25, x, y), lambda: g(B, C, D.double(), 20, 25, x, y),
           lambda: g(B, C, D, 20, 25, x[:3], y), lambda: g(B, C, D, 20, 25, x, y[:, :19].contiguous()),
           lambda: g(B, C, D, 20, 25, x.half(), y), lambda: g(B, C, D, 20, 25, x, y.half()),
           lambda: g(B, C, D, 20, 25, None, y), lambda: g(B, C, D, 20, 25, x, y, False, False),
           lambda: g(B, C, D, 20, 25, x.cpu(), y), lambda: g(B, C, D, 20, 25, x, y, out=(x, None)),
           lambda: g(B, C, D, 20, 25, x, y, out=(y, D)), lambda: g(B, C, D, 20, 25, x[0], y),
           lambda: g(B, C, D, 20, 25, x, y[None])]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")


def test_repairing_a_factored_head():
    """A head's matrix is decomposed; its 8-bit form teaches the factored one: teacher logits by
    apply_quantized, the student's by apply_factors, their distillation, and the gradient of D and of
    the inputs, against the same chain in 64 bits and against differences."""
    rng = np.random.default_rng(12)
    V, n, tokens, top, T = 500, 96, 40, 24, 2.0
    A = (rng.standard_normal((V, n)) * 0.3).astype(np.float32)
    r = erm.decompose(torch.from_numpy(A).cuda(), 1.5, block=16)
    k = r["k"]
    X = torch.from_numpy(rng.standard_normal((tokens, n)).astype(np.float32)).cuda()
    Wq, sw = erm.quantize_rows(torch.from_numpy(A).cuda())
    teacher, index = torch.topk(erm.apply_quantized(Wq, sw, X), top, dim=1)
    w = torch.full((tokens,), 1.0 / tokens, device="cuda")
    w[5] = 0
    Z = erm.apply_factors(r["B"], r["C"], r["D"], V, n, X)
    loss, stats, dZ = erm.distill_loss(Z, teacher, index, T, w, grad=True)
    dX, dD = erm.apply_factors_grad(r["B"], r["C"], r["D"], V, n, X, dZ)

    B = torch.from_numpy(erm.unpack(r["B"], V).astype(np.float64))
    C = torch.from_numpy(erm.unpack(r["C"], n).astype(np.float64))
    x, a, i, wt = X.cpu().double(), teacher.cpu().double(), index.cpu(), w.cpu().double()

    def total(d, xx):
        z = (xx @ C.t() * d) @ B
        logq = torch.log_softmax(z / T, 1).gather(1, i)
        p = torch.softmax(a / T, 1)
        return (wt * T * T * (p * (p.log() - logq)).sum(1)).sum()

    d = r["D"].cpu().double().requires_grad_()
    xx = x.clone().requires_grad_()
    f = total(d, xx)
    f.backward()
    f = f.detach()
    # each step is good to a few 2^-24 of its terms; the chain's logits reach some tens
    assert abs(float(loss.double().sum().cpu() - f)) <= 1e-4 * float(f)
    for got, want in ((dD.cpu().double(), d.grad), (dX.cpu().double(), xx.grad)):
        assert (got - want).norm() <= 1e-4 * want.norm()
    assert not dX[5].any()
    h, v = 1e-4, torch.from_numpy(rng.standard_normal(k))
    with torch.no_grad():
        slope = (total(d + h * v, x) - total(d - h * v, x)) / (2 * h)
    # the central difference's own error is h^2 times a third derivative
    assert abs(float(slope - (dD.cpu().double() * v).sum())) <= 1e-3 * float((dD.cpu().double() * v).abs().sum())


@pytest.mark.parametrize("batch", [4, 9, 70, 300, 4300])
def test_a_bad_vector_gives_nan(batch):
    """The same on every way through the kernels: a NaN or an infinity in dY gives its vector of dX NaN, one
    in X or dY all of dD, one in D all of dX; the rest is untouched."""
    k, m, n = 130, 75, 93
    Bt, Ct, D, X, dY, dX, dD = run(k, m, n, batch, seed=6)
    f = device(Bt, Ct, D)
    for v in (np.inf, -np.inf, np.nan):
        badX, badY = X.copy(), dY.copy()
        badX[1, 5], badY[batch - 1, 7] = v, v
        Xc, Yc, bX, bY = (torch.from_numpy(t).cuda() for t in (X, dY, badX, badY))
        got = erm.apply_factors_grad(*f, m, n, bX, Yc)
        assert torch.equal(got[0], dX) and torch.isnan(got[1]).all()
        got = erm.apply_factors_grad(*f, m, n, Xc, bY)
        assert torch.equal(got[0][:-1], dX[:-1]) and torch.isnan(got[0][-1]).all() and torch.isnan(got[1]).all()
        got = erm.apply_factors_grad(*f, m, n, None, bY, need_dD=False)
        assert torch.equal(got[0][:-1], dX[:-1]) and torch.isnan(got[0][-1]).all()
        assert torch.isnan(erm.apply_factors_grad(*f, m, n, Xc, bY, need_dX=False)[1]).all()
        bad = f[2].clone()
        bad[3] = v
        got = erm.apply_factors_grad(*f[:2], bad, m, n, Xc, Yc)
        assert torch.isnan(got[0]).all() and torch.equal(got[1], dD)


def test_missing_tensors_are_refused():
    B, C, D = device(*random_factors(np.random.default_rng(1), 30, 20, 25))
    x, y = torch.zeros((4, 25), device="cuda"), torch.zeros((4, 20), device="cuda")
    for f in ((None, C, D), (B, None, D), (B, C, None)):
        with pytest.raises(ValueError):
            erm.apply_factors_grad(*f, 20, 25, x, y)
    with pytest.raises(ValueError):
        erm.apply_factors_grad(B, C, D, 20, 25, x, None)


@pytest.mark.parametrize("batch", [4, 300, 4300])
def test_outputs_in_place_and_over_inputs(batch):
    """dX may take the vectors' place, on every way through the kernels; other overlaps are refused."""
    Bt, Ct, D, X, dY, dX, dD = run(130, 93, 93, batch, seed=6)
    f = device(Bt, Ct, D)
    for place in (0, 1):
        v = [torch.from_numpy(t).cuda() for t in (X, dY)]
        got = erm.apply_factors_grad(*f, 93, 93, *v, out=(v[place], torch.empty_like(dD)))
        assert got[0] is v[place] and torch.equal(got[0], dX) and torch.equal(got[1], dD)
    room = torch.zeros(batch * 93 + 93, device="cuda")
    Xc, late = room[:-93].view(batch, 93), room[93:].view(batch, 93)
    Yc = torch.from_numpy(dY).cuda()
    for out in ((late, torch.empty_like(dD)), (torch.empty_like(dX), f[2]), (room[:-93].view(batch, 93), room[-130:])):
        with pytest.raises(erm.ExterndError) as e:
            erm.apply_factors_grad(*f, 93, 93, Xc, Yc, out=out)
        assert e.value.status == erm.EINVAL


def test_every_entry_on_a_stream_of_its_own():
    """The chain of a repair step on a side stream, plain and captured, as on the current one."""
    Bt, Ct, D, X, dY, _, _ = run(130, 75, 93, 40, seed=9)
    f = device(Bt, Ct, D)
    Xc = torch.from_numpy(X).cuda()

    def chain(stream=None):
        q, s = erm.quantize_rows(Xc, stream=stream)
        W, sw = erm.quantize_rows(torch.ones((75, 93), device="cuda").cumsum(1), stream=stream) if stream is None else weights
        teacher = erm.apply_quantized(W, sw, q, s, stream=stream)
        Z = erm.apply_factors_static(*f, 75, 93, Xc, stream=stream)
        loss, stats, d = erm.distill_loss(Z, teacher[:, :20].contiguous(), index, 2.0, grad=True, stream=stream)
        d2 = erm.distill_grad(Z, stats, teacher[:, :20].contiguous(), index, 2.0, stream=stream)
        return (q, s, loss, stats, d, d2, *erm.apply_factors_grad(*f, 75, 93, Xc, d, stream=stream))

    index = torch.arange(20, dtype=torch.int32, device="cuda").repeat(40, 1)
    weights = erm.quantize_rows(torch.ones((75, 93), device="cuda").cumsum(1))
    want = chain()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = chain(side)
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain(torch.cuda.current_stream())
    for _ in range(3):
        for x in got:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)
        assert torch.equal(chain()[6], want[6])
