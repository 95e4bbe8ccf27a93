"""4-bit weights with group scales and products with them against their definitions in 64 bits.

Tolerances.  Codes are compared for equality: a quotient of fp64 rounds as defined.  Products are compared for
equality where every sum is exact in fp32 (whole numbers in X, powers of two as scales, all sums below 2^24 of the
smallest step: then no order of adding rounds).  Elsewhere a sum of n terms in fp32, each of them at most
(55 |s| + |o|) |x| if codes enter as c + 24 and the excess is taken off again, is off by at most n 2^-23 times the sum
of these, and the result rounds once to Y's type (half an eps, and half its smallest step)."""

import pytest
import torch

import expanded_rank_matrix_amd as erm

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def gen(*key):
    return torch.Generator().manual_seed(sum(k * p for k, p in zip(key, (1, 7, 131, 1709, 15551))))


def codes(Q, n):
    c = (Q.cpu()[:, :, None] >> (4 * torch.arange(8, dtype=torch.int32))) & 15
    return (c - 16 * (c >> 3)).reshape(Q.shape[0], -1)[:, :n]


def packed(c, group):
    """Codes (m x n, -8 .. 7) to words; codes behind the rows' ends are arbitrary."""
    m, n = c.shape
    full = torch.full((m, (n + group - 1) // group * group), 5, dtype=torch.int64)
    full[:, :n] = c
    w = ((full & 15).view(m, -1, 8) << (4 * torch.arange(8))).sum(2)
    return torch.where(w >= 2**31, w - 2**32, w).to(torch.int32)


def spread(s, group, n):
    return s.double().repeat_interleave(group, dim=1)[:, :n]


def quantized(w, group, offsets):
    """(codes, scale, offset) by the definition, in 64 bits on the CPU."""
    w = w.cpu().double()
    rows, n = w.shape
    groups = (n + group - 1) // group
    c, s, o = torch.zeros((rows, n)), torch.zeros((rows, groups), dtype=torch.float64), torch.zeros((rows, groups), dtype=torch.float64)
    for g in range(groups):
        v = w[:, g * group:(g + 1) * group]
        if offsets:
            lo, d = v.amin(1, keepdim=True), v.amax(1, keepdim=True) - v.amin(1, keepdim=True)
            q = torch.round(15 * (v - lo) / torch.where(d > 0, d, 1.0)) - 8
            c[:, g * group:(g + 1) * group] = torch.where(d > 0, q, 0.0).float()
            s[:, g], o[:, g] = (d / 15)[:, 0], (lo + 8 * (d / 15))[:, 0]
        else:
            a = v.abs().amax(1, keepdim=True)
            c[:, g * group:(g + 1) * group] = torch.round(7 * v / torch.where(a > 0, a, 1.0)).float()
            s[:, g] = (a.float() / 7).double()[:, 0]
    return c.to(torch.int32), s.float(), o.float()


@pytest.mark.parametrize("offsets", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,n", [(1, 1), (3, 7), (2, 31), (5, 64), (4, 129), (3, 1000), (2, 2560), (70, 333), (1, 40001)])
def test_quantize_matches_definition(rows, n, dtype, group, offsets):
    w = torch.randn((rows, n), generator=gen(rows, n, group)).to(TYPES[dtype])
    for sd in TYPES.values():
        Q, s, o = erm.quantize_groups(w.cuda(), group, offsets, scale_dtype=sd)
        c, ws, wo = quantized(w, group, offsets)
        words = (n + group - 1) // group * group
        assert torch.equal(codes(Q, n), c) and not codes(Q, words)[:, n:].any()
        assert s.dtype == sd and torch.equal(s.cpu(), ws.to(sd))
        assert (o is None) == (not offsets)
        if offsets:
            assert torch.equal(o.cpu(), wo.to(sd))


@pytest.mark.parametrize("offsets", [False, True])
def test_quantize_borders_and_extremes(offsets):
    base = torch.zeros((9, 128))
    base[1] = torch.arange(128) % 15 - 7.0
    base[2] = (torch.arange(128) % 15 - 7.0) / 2  # ties
    base[2, 0] = 7.0
    base[3] = torch.linspace(-1, 1, 128) * 3.4e38
    base[4] = torch.linspace(-1, 1, 128) * 2.0**-126
    base[5] = torch.linspace(-1, 1, 128) * 2.0**-140
    base[6] = 0.25
    base[7] = torch.linspace(1, 1 + 2.0**-20, 128)
    base[8] = torch.randn(128, generator=gen(3)) * 2.0**-90
    Q, s, o = erm.quantize_groups(base.cuda(), 128, offsets)
    c, ws, wo = quantized(base, 128, offsets)
    assert torch.equal(codes(Q, 128), c) and torch.equal(s.cpu(), ws)
    assert not offsets or torch.equal(o.cpu(), wo)
    for bad in (float("nan"), float("inf"), -float("inf")):
        w = torch.randn((2, 300), generator=gen(4))
        w[1, 140] = bad
        Q, s, o = erm.quantize_groups(w.cuda(), 64, offsets)
        k = codes(Q, 300)
        assert torch.isnan(s[1, 2]) and not k[1, 128:192].any() and (not offsets or torch.isnan(o[1, 2]))
        w[1, 128:192] = 0
        c, ws, _ = quantized(w, 64, offsets)
        ok = torch.ones_like(ws, dtype=torch.bool)
        ok[1, 2] = False
        assert torch.equal(s.cpu()[ok], ws[ok]) and torch.equal(k[0], c[0]) and torch.equal(k[1, :128], c[1, :128])
        assert torch.equal(k[1, 192:], c[1, 192:])


def test_quantize_strided_rows_and_given_outputs():
    room = torch.randn((6, 301), generator=gen(9)).to(torch.bfloat16).cuda()
    w = room[:, 3:203]
    want = erm.quantize_groups(w.contiguous(), 64, True)
    out = (torch.empty((6, 32), dtype=torch.int32, device="cuda"), torch.empty((6, 4), device="cuda"), torch.empty((6, 4), device="cuda"))
    got = erm.quantize_groups(w, 64, True, out=out)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1].bfloat16(), want[1]) and torch.equal(got[2].bfloat16(), want[2])


def exact_inputs(tokens, n, m, group, xd, sd, offsets, seed=0):
    """Whole X of -3 .. 3, scales 2^-2 .. 2^2, offsets of -8 .. 8 quarters: every sum is below 2^22 quarters for
    n <= 10000 (|w x| at most 4 (8 + ...) 3), so exact in any order."""
    g = gen(tokens, n, m, group, seed)
    c = torch.randint(-8, 8, (m, n), generator=g)
    groups = (n + group - 1) // group
    s = 2.0 ** torch.randint(-2, 2, (m, groups), generator=g).float()
    o = torch.randint(-8, 9, (m, groups), generator=g).float() / 4 if offsets else None
    x = torch.randint(-3, 4, (tokens, n), generator=g).float()
    return c, s.to(TYPES[sd]), None if o is None else o.to(TYPES[sd]), x.to(TYPES[xd])


def product(c, s, o, x, group):
    w = c.double() * spread(s, group, c.shape[1])
    if o is not None:
        w = w + spread(o, group, c.shape[1])
    return x.double() @ w.t(), w


CASES = [(1, 1, 1), (1, 31, 3), (2, 32, 16), (1, 128, 17), (3, 200, 40), (5, 1000, 33), (1, 2560, 130), (8, 777, 50), (16, 640, 64),
         (17, 129, 70), (31, 520, 20), (33, 300, 100), (64, 1024, 48), (65, 384, 129), (100, 1021, 65), (129, 257, 200), (300, 160, 300),
         (257, 2100, 140)]


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("offsets", [False, True])
@pytest.mark.parametrize("xd,sd", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f16")])
@pytest.mark.parametrize("tokens,n,m", CASES)
def test_products_of_whole_numbers_are_exact(tokens, n, m, xd, sd, offsets, group):
    c, s, o, x = exact_inputs(tokens, n, m, group, xd, sd, offsets)
    y = erm.apply_grouped(packed(c, group).cuda(), s.cuda(), x.cuda(), offset=None if o is None else o.cuda(), group=group,
                          out_dtype=torch.float32)
    assert torch.equal(y.cpu().double(), product(c, s, o, x, group)[0])


@pytest.mark.parametrize("xd", TYPES)
@pytest.mark.parametrize("tokens,n,m", [(1, 9728, 20), (9, 4200, 17), (16, 5000, 33), (40, 4230, 20)])
def test_long_rows_are_exact(tokens, n, m, xd):
    """Rows of several turns of the workgroup's waves."""
    c, s, o, x = exact_inputs(tokens, n, m, 32, xd, "f16", True)
    y = erm.apply_grouped(packed(c, 32).cuda(), s.cuda(), x.cuda(), offset=o.cuda(), group=32, out_dtype=torch.float32)
    assert torch.equal(y.cpu().double(), product(c, s, o, x, 32)[0])


@pytest.mark.parametrize("xd", TYPES)
@pytest.mark.parametrize("tokens", [4, 9, 20, 50])
def test_many_channels_are_exact(tokens, xd):
    c, s, o, x = exact_inputs(tokens, 300, 6200, 64, xd, "bf16", True)
    y = erm.apply_grouped(packed(c, 64).cuda(), s.cuda(), x.cuda(), offset=o.cuda(), group=64, out_dtype=torch.float32)
    w = (c.cuda().double() * spread(s.cuda(), 64, 300) + spread(o.cuda(), 64, 300)).t().contiguous()
    assert torch.equal(y.double(), x.cuda().double() @ w)


def check(tokens, n, m, group, xd, yd, offsets, seed=0, scale=1.0):
    g = gen(tokens, n, m, group, seed)
    c = torch.randint(-8, 8, (m, n), generator=g)
    groups = (n + group - 1) // group
    s = torch.rand((m, groups), generator=g) * 0.01
    o = torch.randn((m, groups), generator=g) * 0.02 if offsets else None
    x = (torch.randn((tokens, n), generator=g) * scale).to(TYPES[xd])
    y = erm.apply_grouped(packed(c, group).cuda(), s.cuda(), x.cuda(), offset=None if o is None else o.cuda(), group=group,
                          out_dtype=TYPES[yd])
    want, _ = product(c, s, o, x, group)
    most = 55 * spread(s, group, n) + (spread(o, group, n).abs() if offsets else 0)
    f = torch.finfo(TYPES[yd])
    half = f.eps / 2 if yd != "f32" else 0.0
    fp32 = n * 2.0**-23 * (x.double().abs() @ most.t())
    tol = fp32 * (1 + half) + want.abs() * (half + 2.0**-24) + f.smallest_normal * f.eps / 2
    off = (y.cpu().double() - want).abs()
    assert not torch.isnan(y).any() and float((off / tol).max()) <= 1.0


@pytest.mark.parametrize("yd", TYPES)
@pytest.mark.parametrize("xd", TYPES)
@pytest.mark.parametrize("tokens,n,m,group,offsets", [(1, 777, 100, 32, True), (4, 2560, 64, 128, False), (20, 500, 90, 64, True),
                                                      (90, 1300, 75, 128, True), (200, 640, 260, 32, False), (1000, 333, 128, 64, True)])
def test_products_match_definition(tokens, n, m, group, offsets, xd, yd):
    check(tokens, n, m, group, xd, yd, offsets)


@pytest.mark.parametrize("tokens", [1, 12, 70, 300])
def test_fp32_tokens_keep_their_bits(tokens):
    """One weight of 1 a channel: Y is X's element, all 24 bits of it."""
    n, m = 256, 256
    c = torch.eye(n, dtype=torch.int64)
    x = torch.randn((tokens, n), generator=gen(tokens))
    y = erm.apply_grouped(packed(c, 32).cuda(), torch.ones((m, n // 32)).cuda(), x.cuda(), group=32)
    # c + 24 and the excess taken off: 25 x and 24 sums of 32 elements, fp32
    tol = 64 * 2.0**-23 * 55 * x.abs().double().view(tokens, -1, 32).sum(2).repeat_interleave(32, dim=1)
    assert ((y.cpu().double() - x.double()).abs() <= tol).all()
    alone = torch.zeros((tokens, n))
    alone[:, ::32] = x[:, ::32]
    y = erm.apply_grouped(packed(c, 32).cuda(), torch.ones((m, n // 32)).cuda(), alone.cuda(), group=32)
    assert ((y.cpu().double() - alone.double()).abs() <= 55 * 2.0**-22 * alone.abs().double().view(tokens, -1, 32).sum(2).repeat_interleave(32, dim=1)).all()


@pytest.mark.parametrize("tokens", [1, 5, 40, 200])
@pytest.mark.parametrize("xd", TYPES)
def test_strided_rows_odd_addresses_and_room_around_the_output(tokens, xd):
    n, m, group = 333, 45, 64
    c, s, o, x = exact_inputs(tokens, n, m, group, xd, "f32", True)
    Q = packed(c, group)
    q = torch.full((m, Q.shape[1] + 3), -1, dtype=torch.int32)
    q[:, 2:-1] = Q
    xs = torch.full((tokens, n + 9), 99.0).to(TYPES[xd])
    xs[:, 5:5 + n] = x
    room = torch.full((tokens, m + 7), 7.0, dtype=torch.float32, device="cuda")
    erm.apply_grouped(q.cuda()[:, 2:-1], s.cuda(), xs.cuda()[:, 5:5 + n], offset=o.cuda(), group=group, out=room[:, 3:3 + m])
    assert torch.equal(room[:, 3:3 + m].cpu().double(), product(c, s, o, x, group)[0])
    assert (room[:, :3] == 7).all() and (room[:, 3 + m:] == 7).all()


@pytest.mark.parametrize("tokens", [1, 20, 150])
def test_one_vector_no_tokens_and_row_results(tokens):
    c, s, o, x = exact_inputs(tokens, 200, 30, 32, "bf16", "bf16", True)
    Q = packed(c, 32).cuda()
    y = erm.apply_grouped(Q, s.cuda(), x.cuda(), offset=o.cuda(), group=32)
    one = erm.apply_grouped(Q, s.cuda(), x[0].cuda(), offset=o.cuda(), group=32)
    assert one.shape == (30,) and torch.equal(one, y[0]) and y.dtype == torch.bfloat16
    assert erm.apply_grouped(Q, s.cuda(), x[:0].cuda(), offset=o.cuda(), group=32).shape == (0, 30)


@pytest.mark.parametrize("tokens", [1, 3, 40, 300])
def test_bad_values_stay_in_their_rows(tokens):
    c, s, o, x = exact_inputs(tokens, 300, 60, 64, "f32", "f32", True)
    x[tokens - 1, 299] = float("nan")
    s[7, 1] = float("nan")
    y = erm.apply_grouped(packed(c, 64).cuda(), s.cuda(), x.cuda(), offset=o.cuda(), group=64).cpu()
    bad = torch.zeros((tokens, 60), dtype=torch.bool)
    bad[tokens - 1], bad[:, 7] = True, True
    assert torch.equal(torch.isnan(y), bad)
    x[tokens - 1, 299], s[7, 1] = 0.0, 1.0
    assert torch.equal(y[~bad].double(), product(c, s, o, x, 64)[0][~bad])


def test_extreme_tokens():
    """fp32 tokens near the ends of their range, where pieces of them are the smallest numbers or near overflow."""
    n, m = 64, 40
    c, s, _, _ = exact_inputs(3, n, m, 32, "f32", "f32", False)
    x = torch.randn((3, n), generator=gen(77))
    x[1] *= 2.0**110
    x[2] *= 2.0**-118
    y = erm.apply_grouped(packed(c, 32).cuda(), s.cuda(), x.cuda(), group=32)
    want, w = product(c, s, None, x, 32)
    tol = n * 2.0**-23 * 55 * (x.double().abs() @ spread(s, 32, n).t()) + n * 55 * 2.0**-126
    assert ((y.cpu().double() - want).abs() <= tol).all()


def test_streams_graphs_and_repeats():
    c, s, o, x = exact_inputs(70, 640, 300, 128, "bf16", "bf16", True)
    Q, s, o, x = packed(c, 128).cuda(), s.cuda(), o.cuda(), x.cuda()
    want = erm.apply_grouped(Q, s, x, offset=o)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [erm.apply_grouped(Q, s, x[:k], offset=o, stream=st) for k, st in zip((70, 1), streams)]
        torch.cuda.synchronize()
        assert torch.equal(got[0], want) and torch.equal(got[1], want[:1])
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        erm.apply_grouped(Q, s, x, offset=o)
    torch.cuda.synchronize()
    graphs, ys = [], []
    for k in (1, 10, 70):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ys.append(erm.apply_grouped(Q, s, x[:k], offset=o))
        graphs.append(g)
    for seed in range(3):
        x.copy_(exact_inputs(70, 640, 300, 128, "bf16", "bf16", True, seed + 1)[3])
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for k, y in zip((1, 10, 70), ys):
            assert torch.equal(y, erm.apply_grouped(Q, s, x[:k], offset=o))


def test_offsets_past_32_bits():
    """Rows of Q 2^20 words apart: the last lies past 2^32 bytes."""
    c, s, o, x = exact_inputs(3, 200, 1100, 64, "bf16", "f32", True)
    Q = packed(c, 64)
    room = torch.empty(1100 << 20, dtype=torch.int32, device="cuda")
    far = room.as_strided((1100, Q.shape[1]), (1 << 20, 1))
    far.copy_(Q)
    for k in (1, 3):
        y = erm.apply_grouped(far, s.cuda(), x[:k].cuda(), offset=o.cuda(), group=64, out_dtype=torch.float32)
        assert torch.equal(y.cpu().double(), product(c, s, o, x[:k], 64)[0])
    big = torch.cat([x] * 40)
    y = erm.apply_grouped(far, s.cuda(), big.cuda(), offset=o.cuda(), group=64, out_dtype=torch.float32)
    assert torch.equal(y.cpu().double(), product(c, s, o, big, 64)[0])


@pytest.mark.parametrize("tokens", [2, 90])
def test_rows_of_codes_too_far_apart_for_a_tile(tokens):
    """2^23 words between rows: a tile's offsets would pass 32 bits."""
    c, s, o, x = exact_inputs(tokens, 200, 20, 64, "bf16", "f32", True)
    Q = packed(c, 64)
    room = torch.empty(20 << 23, dtype=torch.int32, device="cuda")
    far = room.as_strided((20, Q.shape[1]), (1 << 23, 1))
    far.copy_(Q)
    y = erm.apply_grouped(far, s.cuda(), x.cuda(), offset=o.cuda(), group=64, out_dtype=torch.float32)
    assert torch.equal(y.cpu().double(), product(c, s, o, x, 64)[0])


@pytest.mark.parametrize("tokens", [1, 30, 90])
def test_smallest_fp16_tokens_count(tokens):
    """Multiples of fp16's smallest number, 2^-24: whole numbers once scaled, so the products are exact."""
    c, s, o, x = exact_inputs(tokens, 300, 50, 32, "f16", "f32", True)
    y = erm.apply_grouped(packed(c, 32).cuda(), s.cuda(), (x.float() * 2.0**-24).half().cuda(), offset=o.cuda(), group=32, out_dtype=torch.float32)
    assert torch.equal(y.cpu().double() * 2.0**24, product(c, s, o, x, 32)[0])


@pytest.mark.parametrize("xd,tokens", [("bf16", 16384 + 30), ("f32", 16384 + 100)])
def test_more_tokens_than_a_run(xd, tokens):
    c, s, o, x = exact_inputs(tokens, 70, 40, 32, xd, "f16", True)
    y = erm.apply_grouped(packed(c, 32).cuda(), s.cuda(), x.cuda(), offset=o.cuda(), group=32, out_dtype=torch.float32)
    assert torch.equal(y.cpu().double(), product(c, s, o, x, 32)[0])


@pytest.mark.parametrize("xd", TYPES)
def test_whole_rounds_of_tiles_and_tiles_in_parts(xd):
    """More tiles than the card holds at once (512), a last round of some."""
    tokens, m = (1100, 8200) if xd != "f32" else (500, 8300)
    c, s, o, x = exact_inputs(tokens, 520, m, 64, xd, "f32", True)
    y = erm.apply_grouped(packed(c, 64).cuda(), s.cuda(), x.cuda(), offset=o.cuda(), group=64, out_dtype=torch.float32)
    w = (c.cuda().double() * spread(s.cuda(), 64, 520) + spread(o.cuda(), 64, 520)).t().contiguous()
    assert torch.equal(y.double(), x.cuda().double() @ w)


def test_binding_refusals():
    Q, s, o = erm.quantize_groups(torch.randn((8, 100)).cuda(), 32, True)
    x = torch.randn((3, 100)).cuda()
    ok = lambda **k: erm.apply_grouped(**{**dict(Q=Q, scale=s, X=x, offset=o, group=32), **k})  # noqa: E731
    assert ok().shape == (3, 8)
    for bad in (dict(X=x.cpu()), dict(X=x.double()), dict(X=x[:, :90]), dict(X=x.t()), dict(Q=Q[:, :10]), dict(Q=Q.float()), dict(scale=s[:, :2]),
                dict(scale=s.t()), dict(offset=o.half()), dict(offset=o[:4]), dict(group=16), dict(group=64), dict(out_dtype=torch.float64),
                dict(out=torch.empty((3, 7), device="cuda")), dict(out=torch.empty((3, 8), device="cuda"), out_dtype=torch.float16),
                dict(Q=None), dict(scale=None), dict(X=None)):
        with pytest.raises(ValueError):
            ok(**bad)
    with pytest.raises(erm.ExterndError):
        ok(out=x[:, :8])
    w = torch.randn((8, 100)).cuda()
    for bad in (dict(W=w.cpu()), dict(W=w.t()), dict(W=w.int()), dict(group=48), dict(scale_dtype=torch.int8), dict(out=(Q, s, o)),
                dict(out=(Q, s, None), offsets=True), dict(out=(Q, None, None)), dict(W=None)):
        with pytest.raises(ValueError):
            erm.quantize_groups(**{**dict(W=w, group=32), **bad})
