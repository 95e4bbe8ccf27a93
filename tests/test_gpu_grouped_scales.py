"""Scales and offsets of the 4-bit products that the other tests' small powers of two do not tell from their neighbours: the
largest numbers, infinities, and those whose bits only fp32 holds.

Codes enter as c + 8, 0 .. 15, and the excess 8 sum x is taken off.  Where one element of a group is not zero, and x is a
whole number of at most 20 bits, the sums are below 2^24 and the group's whole share c x is exact; what is left is
the product with the scale and the sum over the groups."""

import pytest
import torch

import expanded_rank_matrix_amd as erm

from .test_gpu_grouped import TYPES, gen, packed, product

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
