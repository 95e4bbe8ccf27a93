"""NaN and infinities in the token loss's rows and words: where they show, and that they show nowhere else."""

import pytest
import torch

import expanded_rank_matrix_amd as erm

from .test_gpu_token import TYPES, definition, inputs, near

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("rows", [1, 40, 300])
def test_a_bad_row_has_bad_statistics(rows, value, dtype):
    x, w, target, weight = inputs(rows, 64, 333, TYPES[dtype])
    at = rows // 3
    x[at, 5] = value
    loss, stats, dX, dW = erm.token_loss(x, w, target, weight=weight, grad=True)
    rest = torch.arange(rows, device="cuda") != at
    assert torch.isnan(loss[at]) and torch.isnan(stats[at]).all() and torch.isnan(dX[at]).all() and torch.isnan(dW).all()
    clean = x.clone()
    clean[at] = 0
    want, tol = definition(clean, w, target, weight)
    for a, b, c, name in zip((loss, stats, dX), want, tol, ("loss", "stats", "dX")):
        near(a[rest], b[rest], c[rest], name)
    again = erm.token_grad(x, w, stats, target, grad_loss=weight)
    assert torch.isnan(again[0][at]).all() and torch.isnan(again[1]).all() and torch.equal(again[0][rest], dX[rest])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [3, 200])
def test_a_bad_word_shows_in_every_row(rows, dtype):
    x, w, target, weight = inputs(rows, 40, 700, TYPES[dtype])
    w[600, 7] = NAN
    for out in erm.token_loss(x, w, target, weight=weight, grad=True):
        assert torch.isnan(out).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_an_infinite_word_acts_by_its_logits(dtype):
    rows, vocab, v, j = 64, 500, 300, 9
    x, w, target, weight = inputs(rows, 48, vocab, TYPES[dtype])
    target[target == v] = 0
    x[:, j] = torch.where(x[:, j] == 0, 1.0, x[:, j])
    w[v, j] = -INF
    none = x[:, j] > 0  # the word's logit is -infinity there, +infinity elsewhere
    loss, stats, dX, dW = erm.token_loss(x, w, target, weight=weight, grad=True)
    assert torch.isnan(loss[~none]).all() and torch.isnan(stats[~none]).all() and torch.isnan(dX[~none]).all()
    assert torch.isnan(dW).all()
    # the others: as if the vocabulary lacked the word
    keep = torch.arange(vocab, device="cuda") != v
    moved = torch.where(target > v, target - 1, target)[none]
    want, tol = definition(x[none], w[keep], moved, weight[none])
    for a, b, c, name in zip((loss, stats), want, tol, ("loss", "stats")):
        near(a[none], b, c, name)
    other = torch.arange(48, device="cuda") != j
    near(dX[none][:, other], want[2][:, other], tol[2][:, other], "dX")
    assert not torch.isfinite(dX[:, j]).any()
    # alone, without the rows that it makes NaN; and as the target
    loss, stats, dX, dW = erm.token_loss(x[none], w, target[none], weight=weight[none], grad=True)
    near(dW[keep], want[3], tol[3], "dW")
    loss, _ = erm.token_loss(x[none][:1], w, torch.tensor([v], device="cuda"))
    assert loss[0] == INF


def test_logits_of_minus_infinity_alone():
    x, w = torch.full((2, 8), -INF, device="cuda"), torch.ones((30, 8), device="cuda")
    x[1] = 1.0
    loss, stats = erm.token_loss(x, w, torch.tensor([3, 4], device="cuda"))
    assert torch.isnan(loss[0]) and stats[0].tolist() == [-INF, 0.0] and stats[1].tolist() == [8.0, 30.0]


@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [50, 1100])
def test_a_bad_weight_leaves_the_other_rows_gradient(rows, dtype, value):
    """Weights of 2^-18: a P of fp16 that carries no power of two falls under its smallest number, 2^-24, for most words,
    while dX, of words 256 times as large, stays far above it."""
    x, w, target, weight = inputs(rows, 64, 400, TYPES[dtype])
    x, w = x / 256, w * 256
    weight *= 2.0**-18
    at = rows // 2
    bad = weight.clone()
    bad[at] = value
    loss, _, dX, dW = erm.token_loss(x, w, target, weight=bad, grad=True)
    assert not torch.isfinite(loss[at]) and not torch.isfinite(dX[at]).any() and not torch.isfinite(dW).any()
    # every sum of P and dX itself are carried by the largest weight but the bad one
    weight[at] = 0
    want, tol = definition(x, w, target, weight)
    rest = torch.arange(rows, device="cuda") != at
    near(loss[rest], want[0][rest], tol[0][rest], "loss")
    near(dX[rest], want[2][rest], tol[2][rest], "dX")
