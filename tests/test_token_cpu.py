"""Refusals of the token loss's entry points before any device work, and their workspace sizes."""

import ctypes

import pytest

import expanded_rank_matrix_amd as erm

F32, F16, BF16, I8 = 0, 1, 2, 3
p = ctypes.c_void_p  # never dereferenced: validation fails first
BASE = dict(X=p(1 << 16), t=F32, rows=4, n=8, ldx=8, W=p(1 << 17), vocab=6, ldw=8, target=p(1 << 18), tb=8, weight=p(1 << 19),
            loss=p(1 << 20), stats=p(1 << 21), dX=p(1 << 22), lddx=8, dW=p(1 << 23), lddw=8, ws=p(1 << 24))


def loss(**k):
    a = {**BASE, **k}
    return erm.load().externd_token_loss(a["X"], a["t"], a["rows"], a["n"], a["ldx"], a["W"], a["vocab"], a["ldw"], a["target"],
                                         a["tb"], a["weight"], a["loss"], a["stats"], a["dX"], a["lddx"], a["dW"], a["lddw"],
                                         a["ws"], None)


def grad(**k):
    a = {**BASE, **k}
    return erm.load().externd_token_grad(a["X"], a["t"], a["rows"], a["n"], a["ldx"], a["W"], a["vocab"], a["ldw"], a["stats"],
                                         a["target"], a["tb"], a["weight"], a["dX"], a["lddx"], a["dW"], a["lddw"], a["ws"], None)


@pytest.mark.parametrize("change, word", [
    (dict(X=None), "null"), (dict(W=None), "null"), (dict(target=None), "null"), (dict(stats=None), "null"),
    (dict(t=I8), "x_type"), (dict(t=-1), "x_type"), (dict(tb=2), "target_bytes"),
    (dict(rows=-1), "rows"), (dict(rows=(1 << 20) + 1), "rows"), (dict(n=0), "n <="),
    (dict(n=(1 << 17) + 1, ldx=1 << 20, ldw=1 << 20, lddx=1 << 20, lddw=1 << 20), "n <="),
    (dict(vocab=0), "vocab"), (dict(vocab=(1 << 24) + 1), "vocab"), (dict(ldx=7), "ldx"), (dict(ldw=7), "ldw"),
    (dict(lddx=7), "lddx"), (dict(lddw=7), "lddw"), (dict(ldw=1 << 41), "ldw"), (dict(ws=None), "workspace"),
    (dict(ws=p((1 << 24) + 8)), "workspace")])
def test_refusals(change, word):
    for entry in (loss, grad):
        assert entry(**change) == erm.EINVAL
        assert word in erm.last_error()


def test_refusals_of_one_direction():
    assert loss(loss=None) == erm.EINVAL and "null" in erm.last_error()
    assert grad(dX=None, dW=None) == erm.EINVAL and "dX or dW" in erm.last_error()


@pytest.mark.parametrize("change", [
    dict(dX=p((1 << 16) + 8)), dict(dX=p((1 << 17) + 100)), dict(dX=p(1 << 18)), dict(dX=p((1 << 19) - 120)),
    dict(dW=p((1 << 16) + 4)), dict(dW=p(1 << 17)), dict(dW=p((1 << 22) + 127)), dict(dX=p(1 << 16), dW=p((1 << 16) + 64)),
    dict(dX=p(1 << 21)), dict(dW=p((1 << 21) - 191))])
def test_overlaps_are_refused(change):
    for entry in (loss, grad):
        assert entry(**change) == erm.EINVAL and "overlap" in erm.last_error()


@pytest.mark.parametrize("change", [dict(loss=p(1 << 16)), dict(loss=p((1 << 21) + 4)), dict(stats=p((1 << 17) - 8)),
                                    dict(stats=p((1 << 18) + 16))])
def test_overlaps_of_loss_and_stats_are_refused(change):
    assert loss(**change) == erm.EINVAL and "overlap" in erm.last_error()


def test_a_gradient_in_the_place_of_x_has_its_distance():
    assert loss(dX=p(1 << 16), lddx=9) == erm.EINVAL and "lddx = ldx" in erm.last_error()


def test_nothing_to_do():
    assert loss(rows=0, X=None, target=None, loss=None, stats=None, dX=None, dW=None, ws=None) == erm.OK
    assert grad(rows=0, X=None, target=None, stats=None, dW=None, ws=None) == erm.OK


def test_workspace_sizes():
    size = erm.load().externd_token_workspace
    w = p(1 << 20)
    assert size(BF16, 0, 64, 100, w, 64, 1, 1, 1) == 0
    for t, es in ((F32, 4), (F16, 2), (BF16, 2)):
        for rows, n, vocab in ((1, 1, 1), (33, 64, 1000), (4096, 2560, 131072), (1 << 20, 64, 1 << 24), (1, 1 << 17, 1 << 24)):
            alone, full = size(t, rows, n, vocab, w, n, 1, 0, 0), size(t, rows, n, vocab, w, n, 1, 1, 1)
            assert rows * n * es < alone <= full
            # far below the logits' size where that is large
            if rows * vocab > 1 << 28:
                assert full < 8 * (rows * n * 4 + rows * (vocab // 16) + (1 << 28))
    for bad in ((4, 1, 1, 1, w, 1), (F32, -1, 1, 1, w, 1), (F32, (1 << 20) + 1, 1, 1, w, 1), (F32, 1, 0, 1, w, 1), (F32, 1, 4, 1, w, 3),
                (F32, 1, 1, 0, w, 1), (F32, 1, 1, (1 << 24) + 1, w, 1)):
        assert size(*bad, 1, 1, 1) == -1


def test_binding_refuses_host_and_missing_tensors():
    torch = pytest.importorskip("torch")
    x, w, t = torch.zeros((2, 8)), torch.zeros((4, 8)), torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError):
        erm.token_loss(x, w, t)
    with pytest.raises(ValueError):
        erm.token_grad(x, w, torch.zeros((2, 2)), t)
    with pytest.raises(ValueError):
        erm.token_loss(None, None, None)
    with pytest.raises(ValueError):
        erm.token_grad(None, None, None, None)
