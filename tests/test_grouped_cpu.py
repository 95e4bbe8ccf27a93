"""Refusals of the 4-bit entry points before any device work, and their workspace sizes."""

import ctypes

import pytest

import expanded_rank_matrix_amd as erm

F32, F16, BF16, I8 = 0, 1, 2, 3
p = ctypes.c_void_p  # never dereferenced: validation fails first
far = [p(k << 16) for k in range(1, 9)]


def quantize(W=far[0], t=F32, rows=4, n=40, ldw=40, group=32, Q=far[1], scale=far[2], offset=far[3], st=F32):
    return erm.load().externd_quantize_groups(W, t, rows, n, ldw, group, Q, scale, offset, st, None)


def product(Q=far[0], scale=far[1], offset=far[2], st=F32, group=32, m=4, n=40, ldq=8, X=far[3], xt=F32, tokens=9, ldx=40, Y=far[4],
            yt=F32, ldy=4, ws=far[5]):
    return erm.load().externd_apply_grouped(Q, scale, offset, st, group, m, n, ldq, X, xt, tokens, ldx, Y, yt, ldy, ws, None)


@pytest.mark.parametrize("change, word", [
    (dict(W=None), "null"), (dict(Q=None), "null"), (dict(scale=None), "null"), (dict(t=I8), "w_type"), (dict(st=I8), "s_type"),
    (dict(t=-1), "w_type"), (dict(group=16), "group"), (dict(group=0), "group"), (dict(rows=-1), "rows"), (dict(rows=(1 << 26) + 1), "rows"),
    (dict(n=0), "n <="), (dict(n=(1 << 20) + 1, ldw=1 << 21), "n <="), (dict(ldw=39), "ldw"), (dict(ldw=1 << 41), "ldw")])
def test_quantize_refusals(change, word):
    assert quantize(**change) == erm.EINVAL and word in erm.last_error()


@pytest.mark.parametrize("change, word", [
    (dict(Q=None), "null"), (dict(scale=None), "null"), (dict(X=None), "null"), (dict(Y=None), "null"), (dict(xt=I8), "x_type"),
    (dict(yt=4), "y_type"), (dict(st=-1), "s_type"), (dict(group=33), "group"), (dict(tokens=-1), "tokens"), (dict(tokens=1 << 31), "tokens"),
    (dict(m=0), "m <="), (dict(m=(1 << 26) + 1, ldy=1 << 27), "m <="), (dict(n=0), "n <="), (dict(n=(1 << 20) + 1, ldq=1 << 21, ldx=1 << 21), "n <="),
    (dict(ldq=7), "ldq"), (dict(ldx=39), "ldx"), (dict(ldy=3), "ldy"), (dict(ldy=1 << 41), "ldy")])
def test_product_refusals(change, word):
    assert product(**change) == erm.EINVAL and word in erm.last_error()


# W 4 rows of 160 bytes (640), Q 4 x 8 words (128), scale and offset 4 x 2 (32)
@pytest.mark.parametrize("change", [dict(Q=p((1 << 16) + 636)), dict(scale=p((1 << 16) - 28)), dict(offset=p((1 << 16) + 4)),
                                    dict(scale=p((2 << 16) + 124)), dict(offset=p((2 << 16) - 28)), dict(offset=p((3 << 16) + 28))])
def test_quantize_overlaps_are_refused(change):
    assert quantize(**change) == erm.EINVAL and "overlap" in erm.last_error()


@pytest.mark.parametrize("at", [(1 << 16) + 127, (2 << 16) + 28, (3 << 16) - 140, (4 << 16) + 1436])
def test_product_overlaps_are_refused(at):
    assert product(Y=p(at)) == erm.EINVAL and "overlap" in erm.last_error()


def test_nothing_to_do():
    assert quantize(rows=0, W=None, Q=None, scale=None, offset=None) == erm.OK
    assert product(tokens=0, X=None, Y=None, ws=None) == erm.OK


def test_workspace_sizes():
    size = erm.load().externd_apply_grouped_workspace
    for t in (F32, F16, BF16):
        assert size(t, 0, 100, 100, 32) == 0 and size(t, 1, 2560, 2560, 128) >= 0 and size(t, 2**31 - 1, 1 << 20, 1 << 26, 128) >= 0
    for bad in ((I8, 1, 1, 1, 32), (F32, -1, 1, 1, 32), (F32, 1, 0, 1, 32), (F32, 1, (1 << 20) + 1, 1, 32), (F32, 1, 1, 0, 32),
                (F32, 1, 1, (1 << 26) + 1, 32), (F32, 1, 1, 1, 31)):
        assert size(*bad) == -1


def test_binding_refuses_host_and_missing_tensors():
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError):
        erm.quantize_groups(torch.zeros((2, 8)))
    with pytest.raises(ValueError):
        erm.apply_grouped(torch.zeros((2, 16), dtype=torch.int32), torch.zeros((2, 1)), torch.zeros(8))
    with pytest.raises(ValueError):
        erm.quantize_groups(None)
    with pytest.raises(ValueError):
        erm.apply_grouped(None, None, None)
