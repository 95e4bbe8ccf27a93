"""The token loss where many rows are gathered, in each shape of tiles that fp32 takes, and what it holds beyond the rounding
of its type: against the definition in 64 bits, with the tolerances that are derived beside it."""

import pytest
import torch

import expanded_rank_matrix_amd as erm

from .test_gpu_token import TYPES, check, definition, inputs, near

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,vocab", [(65, 10007), (300, 32768), (600, 32768), (1024, 32700)])
@pytest.mark.parametrize("n", [68, 61])
def test_fp32_in_tiles_of_every_shape(rows, vocab, n):
    x, w, target, weight = inputs(rows, n, vocab, torch.float32)
    target[1::9] = -100
    check(x, w, target, weight)


def left_out(rows, how):
    """Which rows do not count."""
    r = torch.arange(rows, device="cuda")
    if how == "runs":  # irregular: of 1 to 13 rows, across the blocks of 64 and of 1024
        return ((r * r // 7) % 13 < 5) | ((r >= 1000) & (r < 1030))
    if how == "a block":  # the second 1024 rows, or what there is of them
        return (r >= 1024) & (r < 2048)
    if how == "all but the last":
        return r < rows - 1
    return r % 64 != 63  # one in 64


@pytest.mark.parametrize("how", ["runs", "a block", "all but the last", "one in 64"])
@pytest.mark.parametrize("rows", [1024, 1025, 2050, 4000])
@pytest.mark.parametrize("dtype", TYPES)
def test_many_rows_with_some_left_out(rows, how, dtype):
    """Above 1024 rows the ones that count are found by rounds of 1024 and gathered by a launch of their own."""
    x, w, target, weight = inputs(rows, 56, 333, TYPES[dtype], 3)
    out = left_out(rows, how)
    at = torch.nonzero(out)[:, 0]
    target[at[::2]] = -100
    weight[at[1::2]] = 0.0
    clean = torch.where(out[:, None], 0.0, x)
    x[out] = float("nan")
    want, tol = definition(clean, w, target, weight)
    names = ("loss", "stats", "dX", "dW")
    got = erm.token_loss(x, w, target.int() if rows % 2 else target, weight=weight, grad=True)
    for a, b, c, name in zip(got, want, tol, names):
        near(a, b, c, name)
        if name != "dW":
            assert not a[out].any()
    for a, b in zip(erm.token_loss(x, w, target, weight=weight), got):
        assert torch.equal(a, b)
    for a, b, c, name in zip(erm.token_grad(x, w, got[1], target, grad_loss=weight), want[2:], tol[2:], names[2:]):
        near(a, b, c, name + " alone")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [1025, 3000])
def test_no_row_of_many_counts(rows, dtype):
    x, w, target, weight = inputs(rows, 40, 100, TYPES[dtype])
    x[:] = float("nan")
    target[::2] = -100
    weight[1::2] = 0.0
    got = erm.token_loss(x, w, target, weight=weight, grad=True)
    for t in (*got, *erm.token_grad(x, w, got[1], target, grad_loss=weight)):
        assert not t.any()


@pytest.mark.parametrize("dtype,vocab", [("bf16", 512), ("f16", 4096), ("f32", 512)])
@pytest.mark.parametrize("rows", [1, 40, 1500])
def test_what_the_rounding_of_the_targets_share_takes_comes_back(rows, dtype, vocab):
    """Rows of zeros: every probability is 1 / vocab, a power of two, and the target's P is -(1 - 1 / vocab) g, one bit
    longer than the type holds, so rounded to -g.  W is 1 + d with small d, in steps of the type: dX is the mean of d less the
    target's, and without what the rounding took it would be off by g / vocab, many times that.  All sums are exact in fp32."""
    dt = TYPES[dtype]
    n, step = 24, 2.0**-7 if dtype == "bf16" else 2.0**-10
    g = torch.Generator().manual_seed(rows + vocab)
    d = torch.randint(0, 3, (vocab, n), generator=g).double().cuda() * step
    w = (1 + d).to(dt)
    assert torch.equal(w.double(), 1 + d)
    x = torch.zeros((rows, n), dtype=dt, device="cuda")
    target = torch.randint(0, vocab, (rows,), generator=g).cuda()
    weight = (2.0 ** torch.randint(-3, 4, (rows,), generator=g).float()).cuda()
    loss, stats, dX, dW = erm.token_loss(x, w, target, weight=weight, grad=True)
    want = (d.mean(0) - d[target]) * weight.double()[:, None]
    # half a step of the type: relative, but below its smallest normal number (fp16's 2^-14) half of one step there
    f = torch.finfo(dt)
    assert ((dX.double() - want).abs() <= f.eps / 2 * want.abs().clamp(min=f.smallest_normal)).all()
    assert torch.equal(stats, torch.tensor([0.0, float(vocab)], device="cuda").expand(rows, 2)) and not dW.any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("factor", [256.0, 1 / 256])
def test_small_weights_keep_every_element(dtype, factor):
    """Weights of 2^-18, so that most P lie below fp16's smallest number, and rows 256 times as large as words, or the other
    way round, so that one of the gradients does not."""
    x, w, target, weight = inputs(50, 64, 400, TYPES[dtype])
    check(x * factor, w / factor, target, weight * 2.0**-18)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_far_apart(dtype):
    """The last rows of X, dX and dW lie 2^32 bytes and more behind the first, and words 2^24 bytes apart are copied."""
    dt = TYPES[dtype]
    rows, n, vocab = 40, 24, 300
    x, w, target, weight = inputs(rows, n, vocab, dt)
    target[-1], target[-2] = vocab - 1, vocab - 2
    want = erm.token_loss(x, w, target, weight=weight, grad=True)
    wide, far = (1 << 32) // (rows - 1) // dt.itemsize + 3, (1 << 24) // dt.itemsize
    xs = torch.empty(rows * wide, dtype=dt, device="cuda").as_strided((rows, n), (wide, 1))
    ws = torch.empty(vocab * far, dtype=dt, device="cuda").as_strided((vocab, n), (far, 1))
    dx = torch.empty(rows * wide, dtype=dt, device="cuda").as_strided((rows, n), (wide, 1))
    dw = torch.empty(vocab * far, dtype=dt, device="cuda").as_strided((vocab, n), (far, 1))
    xs.copy_(x)
    ws.copy_(w)
    got = erm.token_loss(xs, ws, target, weight=weight, out=(dx, dw))
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("rows,vocab", [(1, 300), (65, 10007), (300, 32768), (600, 32768)])
def test_long_fp32_sums_keep_small_terms(rows, vocab):
    """Logits of 4096 terms of 1 + 2^-14: 4096.25, which fp32 holds, but a sum past 2048 that takes the terms one after the other
    loses the small part of each.  In runs of up to 256 every partial sum is exact (a run 256 + 2^-6, steps of 2^-15)."""
    n = 4096
    x = torch.ones((rows, n), device="cuda")
    w = torch.full((vocab, n), 1 + 2.0**-14, device="cuda")
    loss, stats = erm.token_loss(x, w, torch.zeros(rows, dtype=torch.int64, device="cuda"))
    assert (stats[:, 0] == 4096.25).all() and (stats[:, 1] == vocab).all()
    # the logarithm in fp64, rounded once
    assert ((loss.double() - torch.tensor(float(vocab)).double().log().cuda()).abs() <= 2.0**-23 * 16).all()


def test_long_fp32_sums_over_rows_keep_small_terms():
    """Words of zeros: P is 1 / vocab, and dW of a word that is no target the mean of its rows times their number."""
    rows, n, vocab = 4096, 40, 64
    x = torch.full((rows, n), 1 + 2.0**-14, device="cuda")
    w = torch.zeros((vocab, n), device="cuda")
    _, _, dX, dW = erm.token_loss(x, w, torch.zeros(rows, dtype=torch.int64, device="cuda"), grad=True)
    assert not dX.any() and (dW[1:] == 4096.25 / vocab).all()
