"""Refusals of the distillation entry points before any device work, and their workspace sizes."""

import ctypes

import pytest

import expanded_rank_matrix_amd as erm

fake, other = ctypes.c_void_p(256), ctypes.c_void_p(1 << 20)  # never dereferenced: validation fails first


def loss(z=fake, zt=0, rows=4, vocab=100, ldz=100, t=fake, tt=0, i=fake, ib=4, top=8, T=1.0, w=None, out=fake, stats=fake,
         d=None, ldd=100, ws=fake):
    return erm.load().externd_distill_loss(z, zt, rows, vocab, ldz, t, tt, i, ib, top, T, w, out, stats, d, ldd, ws, None)


def grad(z=fake, zt=0, rows=4, vocab=100, ldz=100, stats=fake, t=fake, tt=0, i=fake, ib=4, top=8, T=1.0, g=None, d=other,
         ldd=100):
    return erm.load().externd_distill_grad(z, zt, rows, vocab, ldz, stats, t, tt, i, ib, top, T, g, d, ldd, None)


COMMON = [(dict(z=None), "null"), (dict(t=None), "null"), (dict(i=None), "null"), (dict(stats=None), "null"),
          (dict(zt=3), "z_type"), (dict(tt=3), "t_type"), (dict(zt=-1), "z_type"), (dict(ib=2), "index_bytes"),
          (dict(rows=-1), "rows"), (dict(rows=1 << 31), "rows"), (dict(vocab=0), "vocab"),
          (dict(vocab=(1 << 30) + 1, ldz=1 << 31), "vocab"), (dict(top=0), "top"), (dict(top=1025), "top"),
          (dict(ldz=99), "ldz"), (dict(T=0.0), "temperature"), (dict(T=-1.0), "temperature"),
          (dict(T=float("nan")), "temperature"), (dict(T=float("inf")), "temperature"), (dict(T=1e-4), "temperature"),
          (dict(d=other, ldd=99), "ldd"), (dict(d=fake, ldd=101), "ldd = ldz")]


@pytest.mark.parametrize("change, word", COMMON + [(dict(out=None), "null"), (dict(vocab=5000, ldz=5000, ws=None), "workspace"),
                                                   (dict(vocab=5000, ldz=5000, ws=ctypes.c_void_p(8)), "workspace")])
def test_loss_refusals(change, word):
    assert loss(**change) == erm.EINVAL
    assert word in erm.last_error()


@pytest.mark.parametrize("change, word", COMMON + [(dict(d=None), "null")])
def test_grad_refusals(change, word):
    assert grad(**change) == erm.EINVAL
    assert word in erm.last_error()


def test_nothing_to_do():
    assert loss(rows=0, z=None, t=None, i=None, out=None, stats=None, ws=None) == erm.OK
    assert grad(rows=0, z=None, t=None, i=None, stats=None, d=None) == erm.OK


def test_workspace_sizes():
    size = erm.load().externd_distill_workspace
    assert size(0, 100) == 0 and size(4096, 131072) == 0
    assert size(1, 131072) > 0
    assert size(-1, 5) == -1 and size(5, 0) == -1 and size(1 << 31, 5) == -1 and size(5, (1 << 30) + 1) == -1


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    z, t, i = torch.zeros((2, 8)), torch.zeros((2, 3)), torch.zeros((2, 3), dtype=torch.int32)
    with pytest.raises(ValueError):
        erm.distill_loss(z, t, i)
    with pytest.raises(ValueError):
        erm.distill_grad(z, torch.zeros((2, 2)), t, i)


@pytest.mark.parametrize("entry, count", [(erm.distill_loss, 3), (erm.distill_grad, 4)])
def test_missing_tensors_are_refused(entry, count):
    with pytest.raises(ValueError):
        entry(*[None] * count)


# 4 rows of 100 fp32 (ldz 100: bytes 65536 .. 67135; ldz 250: rows 1000 bytes apart)
@pytest.mark.parametrize("at, ldz, ldd", [(65540, 100, 100), (67132, 100, 100), (65536 - 1596, 100, 100), (65536 + 400, 100, 100),
                                          (65536 + 396, 250, 250), (65536 - 396, 250, 250), (65536 + 604, 250, 250),
                                          (65536 + 2004, 250, 250), (65536 + 400, 250, 300), (65536, 250, 300)])
def test_gradient_over_the_logits_is_refused(at, ldz, ldd):
    z, d = ctypes.c_void_p(65536), ctypes.c_void_p(at)
    assert loss(z=z, ldz=ldz, d=d, ldd=ldd) == erm.EINVAL and "logits" in erm.last_error()
    assert grad(z=z, ldz=ldz, d=d, ldd=ldd) == erm.EINVAL and "logits" in erm.last_error()
