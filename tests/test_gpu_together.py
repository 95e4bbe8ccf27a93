"""The operators that serve and train a compressed model, run together as such a model uses them: hidden rows through
a factored layer and a layer in 4 bits, tokens answered through an output matrix in 4 bits, and a step of repair from
the tokens' loss back to the factored layer's scales.

Tolerances.  Each operator's own are tested elsewhere; here every value is compared with the whole chain in 64 bits at
the rounding of what passes between the operators: bf16 rows (half a step is 2^-9 of a value) and their products over
n terms, whose errors are independent, so that the 2-norm of a result is off by a few 2^-9 of its own."""

import pytest
import torch

import expanded_rank_matrix_amd as erm

pytestmark = pytest.mark.gpu


def dense(words, length):
    return torch.from_numpy(erm.unpack(words, length)).double().cuda()


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.fixture(scope="module")
def model():
    g = torch.Generator().manual_seed(8)
    m, n, vocab = 192, 128, 700
    A = torch.randn((m, n), generator=g).cuda()
    f = erm.decompose(A, 1.5)
    layer = torch.randn((160, m), generator=g).cuda() * m**-0.5
    head = (torch.randn((vocab, 160), generator=g) * 160**-0.5).to(torch.bfloat16).cuda()
    x = torch.randn((90, n), generator=g).cuda()
    target = torch.randint(0, vocab, (90,), generator=g).cuda()
    target[::7] = -100
    return dict(m=m, n=n, vocab=vocab, f=f, layer=layer, head=head, x=x, target=target)


@pytest.mark.parametrize("group", [32, 128])
def test_serving_through_4_bits(model, group):
    M = model
    f = M["f"]
    Q, s, o = erm.quantize_groups(M["layer"], group, offsets=True)
    HQ, hs, _ = erm.quantize_groups(M["head"], group, scale_dtype=torch.float32)
    h = erm.apply_factors(f["B"], f["C"], f["D"], M["m"], M["n"], M["x"])
    y = erm.apply_grouped(Q, s, h, offset=o, group=group, out_dtype=torch.bfloat16)
    z = erm.apply_grouped(HQ, hs, y, group=group, out_dtype=torch.float32)
    one = erm.apply_grouped(HQ, hs, y[3], group=group, out_dtype=torch.float32)

    def widened(Q, s, o, n):
        c = (Q[:, :, None] >> (4 * torch.arange(8, device="cuda", dtype=torch.int32))) & 15
        w = (c - 16 * (c >> 3)).reshape(len(Q), -1)[:, :n].double() * s.double().repeat_interleave(group, 1)[:, :n]
        return w if o is None else w + o.double().repeat_interleave(group, 1)[:, :n]

    h64 = M["x"].double() @ dense(f["C"], M["n"]).t().contiguous() * f["D"].double() @ dense(f["B"], M["m"])
    w, v = widened(Q, s, o, M["m"]), widened(HQ, hs, None, 160)
    z64 = h64 @ w.t().contiguous() @ v.t().contiguous()
    assert off(h, h64) < 1e-6 and off(y, h64 @ w.t().contiguous()) < 2**-8 and off(z, z64) < 2**-7
    assert off(one, z64[3]) < 2**-7
    # codes and scales hold the weights to half a step of their group
    assert ((w - M["layer"].double()).abs() <= 0.501 * s.double().repeat_interleave(group, 1)[:, :M["m"]]).all()


def test_repair_from_tokens(model):
    """loss(tokens) of head (B diag(D) C x): its gradient at D through token_loss and apply_factors_grad, against 64 bits."""
    M = model
    f = M["f"]
    W = (torch.randn((M["vocab"], M["m"]), generator=torch.Generator().manual_seed(3)) * M["m"]**-0.5).cuda()
    weight = torch.full((90,), 1.0 / 77, device="cuda")
    h = erm.apply_factors(f["B"], f["C"], f["D"], M["m"], M["n"], M["x"])
    for dt, bound in ((torch.float32, 1e-4), (torch.bfloat16, 2**-6)):
        loss, stats, dh, dW = erm.token_loss(h.to(dt), W.to(dt), M["target"], weight=weight, grad=True)
        dX, dD = erm.apply_factors_grad(f["B"], f["C"], f["D"], M["m"], M["n"], M["x"], dh.float())
        x, D, V = M["x"].double().requires_grad_(), f["D"].double().requires_grad_(), W.to(dt).double().requires_grad_()
        h64 = (x @ dense(f["C"], M["n"]).t() * D) @ dense(f["B"], M["m"])
        want = torch.nn.functional.cross_entropy(h64 @ V.t(), M["target"], ignore_index=-100, reduction="none") / 77
        want.sum().backward()
        assert off(loss, want.detach()) < bound and off(dW, V.grad) < bound
        assert off(dX, x.grad) < bound and off(dD, D.grad) < bound
        again = erm.token_grad(h.to(dt), W.to(dt), stats, M["target"], grad_loss=weight, need_dW=False)
        assert torch.equal(again[0], dh) and again[1] is None
