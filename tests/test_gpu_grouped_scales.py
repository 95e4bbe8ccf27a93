"""Scales and offsets of the 4-bit products that the other tests' small powers of two do not tell from their neighbours: the
largest numbers, infinities, and those whose bits only fp32 holds.

Codes enter as c + 8, 0 .. 15, and the excess 8 sum x is taken off.  Where one element of a group is not zero, and x is a
whole number of at most 20 bits, the sums are below 2^24 and the group's whole share c x is exact; what is left is
the product with the scale and the sum over the groups."""

import pytest
import torch

import expanded_rank_matrix_amd as erm

from .test_gpu_grouped import TYPES, exact_inputs, gen, packed, product, spread

pytestmark = pytest.mark.gpu

TOKENS = [1, 20, 64, 65, 300]


@pytest.mark.parametrize("sd", ["f32", "bf16"])
@pytest.mark.parametrize("offsets", [False, True])
@pytest.mark.parametrize("tokens", TOKENS)
def test_the_largest_scales(tokens, sd, offsets):
    """Scales of 2^126 and products that come back into range: 8 s is infinite, s c x is not."""
    n, m, group = 200, 40, 64
    g = gen(tokens, n)
    c = torch.randint(-8, 8, (m, n), generator=g)
    s = torch.full((m, 4), 2.0**126).to(TYPES[sd])
    o = torch.where(torch.rand((m, 4), generator=g) < 0.5, -1.0, 1.0).mul(2.0**126).to(TYPES[sd]) if offsets else None
    x = torch.randint(-3, 4, (tokens, n), generator=g).float() * 2.0**-20
    y = erm.apply_grouped(packed(c, group).cuda(), s.cuda(), x.cuda(), offset=None if o is None else o.cuda(), group=group)
    assert torch.equal(y.cpu().double(), product(c, s, o, x, group)[0])


@pytest.mark.parametrize("tokens", TOKENS)
@pytest.mark.parametrize("where", ["scale", "offset"])
def test_an_infinite_scale_stays_in_its_channel(tokens, where):
    n, m, group = 300, 60, 64
    g = gen(tokens, m)
    c = torch.randint(-8, 8, (m, n), generator=g)
    s, o = torch.ones((m, 5)), torch.ones((m, 5))
    x = torch.randint(1, 4, (tokens, n), generator=g).float()
    (s if where == "scale" else o)[7, 1] = float("inf")
    y = erm.apply_grouped(packed(c, group).cuda(), s.cuda(), x.cuda(), offset=o.cuda(), group=group).cpu()
    rest = torch.arange(m) != 7
    assert not torch.isfinite(y[:, 7]).any()
    want, _ = product(c, s, o, x, group)
    assert torch.equal(y[:, rest].double(), want[:, rest])
    if where == "offset":  # sum x is above 0
        assert (y[:, 7] == float("inf")).all()


def lone(tokens, n, group, values):
    """Tokens with one element that is not zero each, in groups and places that change from token to token."""
    x = torch.zeros((tokens, n))
    t = torch.arange(tokens)
    x[t, (t * 37 + t // 5) % n] = values
    return x


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("tokens", TOKENS)
def test_every_bit_of_fp32_tokens_enters(tokens, group):
    """Odd whole numbers of 20 bits: three pieces of 8.  (c + 8) x is below 2^24, and scales are powers of two: exact."""
    n, m = 300, 50
    g = gen(tokens, n, group)
    c = torch.randint(-8, 8, (m, n), generator=g)
    s = 2.0 ** torch.randint(-3, 4, (m, (n + group - 1) // group), generator=g).float()
    v = (2 * torch.randint(2**18, 2**19, (tokens,), generator=g) + 1).float() * torch.where(torch.rand(tokens, generator=g) < 0.5, -1.0, 1.0)
    x = lone(tokens, n, group, v)
    y = erm.apply_grouped(packed(c, group).cuda(), s.cuda(), x.cuda(), group=group)
    assert torch.equal(y.cpu().double(), product(c, s, None, x, group)[0])


@pytest.mark.parametrize("xd", TYPES)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("tokens", TOKENS)
def test_every_bit_of_fp32_scales_and_offsets_enters(tokens, group, xd):
    """x a power of two.  Offsets alone: the product with one is exact.  Scales: s (c + 8) x and 8 s x, or their difference,
    round at most three times, each of at most 23 |s x|; a scale rounded to 16 bits would be off by up to 2^-12 |s c x| (fp16)."""
    n, m = 300, 50
    g = gen(tokens, m, group)
    groups = (n + group - 1) // group
    c = torch.randint(-8, 8, (m, n), generator=g)
    s, o = torch.rand((m, groups), generator=g) + 0.5, torch.randn((m, groups), generator=g)
    x = lone(tokens, n, group, 2.0 ** torch.randint(-4, 5, (tokens,), generator=g).float())
    Q, X = packed(c, group).cuda(), x.to(TYPES[xd]).cuda()
    y = erm.apply_grouped(Q, torch.zeros_like(s).cuda(), X, offset=o.cuda(), group=group, out_dtype=torch.float32)
    assert torch.equal(y.cpu().double(), product(c, torch.zeros_like(s), o, x, group)[0])
    y = erm.apply_grouped(Q, s.cuda(), X, group=group, out_dtype=torch.float32)
    size = x.double().abs() @ s.double().repeat_interleave(group, 1)[:, :n].t()
    assert ((y.cpu().double() - product(c, s, None, x, group)[0]).abs() <= 3 * 23 * 2.0**-24 * size).all()


@pytest.mark.parametrize("xd", TYPES)
@pytest.mark.parametrize("tokens,m", [(1, 4100), (8, 8190), (8, 8200), (9, 4100), (20, 8200), (50, 4100), (3, 12300), (1, 33000)])
def test_channels_around_whole_rounds_are_exact(tokens, m, xd):
    """Either width of the kernel for few tokens, at sizes where it changes: whole numbers, so that no order of sums rounds."""
    c, s, o, x = exact_inputs(tokens, 300, m, 32, xd, "bf16", True)
    y = erm.apply_grouped(packed(c, 32).cuda(), s.cuda(), x.cuda(), offset=o.cuda(), group=32, out_dtype=torch.float32)
    w = (c.cuda().double() * spread(s.cuda(), 32, 300) + spread(o.cuda(), 32, 300)).t().contiguous()
    assert torch.equal(y.double(), x.cuda().double() @ w)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("tokens", [32, 33, 40, 63, 64, 65])
@pytest.mark.parametrize("n,m", [(70, 33), (1100, 150), (300, 4200)])
def test_fp32_tokens_around_the_border_between_the_kernels(n, m, tokens, group):
    c, s, o, x = exact_inputs(tokens, n, m, group, "f32", "f32", True)
    y = erm.apply_grouped(packed(c, group).cuda(), s.cuda(), x.cuda(), offset=o.cuda(), group=group)
    w = (c.cuda().double() * spread(s.cuda(), group, n) + spread(o.cuda(), group, n)).t().contiguous()
    assert torch.equal(y.double(), x.cuda().double() @ w)
