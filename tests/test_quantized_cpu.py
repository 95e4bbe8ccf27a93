"""Refusals of the 8-bit entry points before any device work, and their workspace sizes."""

import ctypes

import pytest

import expanded_rank_matrix_amd as erm

F32, F16, BF16, I8 = 0, 1, 2, 3
fake = ctypes.c_void_p(256)  # never dereferenced: validation fails first


def quantize(X=fake, t=F32, rows=4, n=8, ldx=8, Q=fake, ldq=8, scale=fake):
    return erm.load().externd_quantize_rows(X, t, rows, n, ldx, Q, ldq, scale, None)


def product(W=fake, sw=fake, m=4, n=8, ldw=8, X=fake, xt=I8, sx=fake, tokens=9, ldx=8, Y=fake, yt=F32, ldy=4, ws=fake):
    return erm.load().externd_apply_quantized(W, sw, m, n, ldw, X, xt, sx, tokens, ldx, Y, yt, ldy, ws, None)


@pytest.mark.parametrize("change, word", [
    (dict(X=None), "null"), (dict(Q=None), "null"), (dict(scale=None), "null"),
    (dict(t=I8), "x_type"), (dict(t=7), "x_type"), (dict(t=-1), "x_type"),
    (dict(rows=-1), "rows"), (dict(rows=1 << 31), "rows"), (dict(n=0), "n <"), (dict(n=1 << 31, ldx=1 << 31, ldq=1 << 31), "n <"),
    (dict(ldx=7), "ldx"), (dict(ldq=7), "ldq"), (dict(ldx=1 << 41), "ldx")])
def test_quantize_refusals(change, word):
    assert quantize(**change) == erm.EINVAL
    assert word in erm.last_error()


@pytest.mark.parametrize("change, word", [
    (dict(W=None), "null"), (dict(sw=None), "null"), (dict(X=None), "null"), (dict(Y=None), "null"),
    (dict(xt=4), "x_type"), (dict(yt=I8), "y_type"), (dict(yt=-1), "y_type"),
    (dict(tokens=-1), "tokens"), (dict(tokens=1 << 31), "tokens"), (dict(m=0), "m <"), (dict(m=(1 << 26) + 1, ldy=1 << 31), "m <"),
    (dict(n=0), "131071"), (dict(n=131072, ldw=131072, ldx=131072), "131071"),
    (dict(ldw=7), "ldw"), (dict(ldx=7), "ldx"), (dict(ldy=3), "ldy"),
    (dict(sx=None), "x_scale"), (dict(xt=BF16), "x_scale"),
    (dict(xt=BF16, sx=None, ws=None), "workspace"), (dict(xt=F32, sx=None, ws=ctypes.c_void_p(264)), "workspace")])
def test_product_refusals(change, word):
    assert product(**change) == erm.EINVAL
    assert word in erm.last_error()


def test_nothing_to_do():
    assert quantize(rows=0, X=None, Q=None, scale=None) == erm.OK
    assert product(tokens=0, X=None, Y=None, ws=None) == erm.OK


def test_workspace_sizes():
    size = erm.load().externd_apply_quantized_workspace
    assert size(I8, 3, 100, 100) == 0
    assert size(BF16, 0, 100, 100) == 0
    for t, n in ((9, 1), (3, 17000), (1000, 131071), (2**31 - 1, 131071)):
        for ty in (F32, F16, BF16):
            assert size(ty, t, n, 1000) >= t * 4 + t * n
    for bad in ((4, 1, 1, 1), (F32, -1, 1, 1), (F32, 1, 0, 1), (F32, 1, 131072, 1), (F32, 1, 1, 0), (F32, 1, 1, (1 << 26) + 1)):
        assert size(*bad) == -1


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    x, w = torch.zeros((2, 8)), torch.zeros((4, 8), dtype=torch.int8)
    with pytest.raises(ValueError):
        erm.quantize_rows(x)
    with pytest.raises(ValueError):
        erm.apply_quantized(w, torch.zeros(4), x)


@pytest.mark.parametrize("entry, count", [(erm.quantize_rows, 1), (erm.apply_quantized, 3)])
def test_missing_tensors_are_refused(entry, count):
    with pytest.raises(ValueError):
        entry(*[None] * count)


@pytest.mark.parametrize("at, ldq", [(65536, 8), (65536 + 127, 8), (65536 - 31, 8), (65536 + 64, 64), (65536 + 33, 40)])
def test_quantize_over_its_rows_is_refused(at, ldq):
    """4 rows of 8 fp32: bytes 65536 .. 65663 (ldx 8), or rows of 32 of every 64 bytes (ldx 16)."""
    p = ctypes.c_void_p
    ldx = 16 if ldq == 64 else 8
    assert quantize(X=p(65536), Q=p(at), ldx=ldx, ldq=ldq, scale=p(1 << 20)) == erm.EINVAL and "overlap" in erm.last_error()
    assert quantize(X=p(1 << 18), Q=p(at), scale=p(at + 20)) == erm.EINVAL and "overlap" in erm.last_error()
    assert quantize(X=p(65536), Q=p(1 << 20), scale=p(65536 + 124)) == erm.EINVAL and "overlap" in erm.last_error()


@pytest.mark.parametrize("at", [65536 + 71, (1 << 17) + 28, (1 << 18) + 12, (1 << 19) + 32, (1 << 17) - 140])
def test_product_over_its_inputs_is_refused(at):
    """9 tokens of 8 codes by 4 channels: X 72 bytes, W 32, its scales 16, the tokens' 36, Y 144."""
    p = ctypes.c_void_p
    rc = product(X=p(65536), W=p(1 << 17), sw=p(1 << 18), sx=p(1 << 19), Y=p(at))
    assert rc == erm.EINVAL and "overlap" in erm.last_error()
