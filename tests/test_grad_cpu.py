"""Refusals of the factored layer's gradient before any device work, and its workspace sizes."""

import ctypes

import pytest

import expanded_rank_matrix_amd as erm

fake = ctypes.c_void_p(256)  # never dereferenced: validation fails first


def grad(B=fake, C=fake, D=fake, k=8, m=4, n=4, X=fake, dY=fake, batch=2, dX=fake, dD=fake, ws=fake):
    return erm.load().externd_apply_factors_grad(B, C, D, k, m, n, X, dY, batch, dX, dD, ws, None)


@pytest.mark.parametrize("change, word", [
    (dict(B=None), "null"), (dict(C=None), "null"), (dict(D=None), "null"), (dict(dY=None), "null"), (dict(X=None), "null"),
    (dict(dX=None, dD=None), "dX or dD"), (dict(k=0), "k, m, n"), (dict(m=0), "k, m, n"), (dict(n=0), "k, m, n"),
    (dict(k=(1 << 23) + 1), "k, m, n"), (dict(k=1 << 20, m=(1 << 13) + 1), "2^33"), (dict(k=1 << 20, n=(1 << 13) + 1), "2^33"), (dict(batch=-1), "batch"), (dict(batch=1 << 31), "batch"),
    (dict(ws=None), "workspace"), (dict(ws=ctypes.c_void_p(8)), "workspace")])
def test_refusals(change, word):
    assert grad(**change) == erm.EINVAL
    assert word in erm.last_error()


def test_nothing_to_do():
    assert grad(batch=0, dX=None, dD=None, dY=None, X=None, ws=None) == erm.OK


def test_workspace_sizes():
    size = erm.load().externd_apply_factors_grad_workspace
    assert size(8, 4, 4, 0) == 0 and size(8, 4, 4, 1) > 0
    assert size(100, 50, 60, 8192) == size(100, 50, 60, 1 << 30)  # passes of bounded size
    for bad in ((0, 1, 1, 1), (1, 0, 1, 1), (1, 1, 0, 1), (1, 1, 1, -1), (1, 1, 1, 1 << 31), ((1 << 23) + 1, 1, 1, 1)):
        assert size(*bad) == -1


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    w = torch.zeros((3, 1), dtype=torch.int32)
    with pytest.raises(ValueError):
        erm.apply_factors_grad(w, w, torch.zeros(3), 4, 4, torch.zeros((2, 4)), torch.zeros((2, 4)))


def test_missing_tensors_are_refused():
    with pytest.raises(ValueError):
        erm.apply_factors_grad(None, None, None, 4, 4, None, None)


@pytest.mark.parametrize("change", [dict(dD=1 << 16), dict(dX=(1 << 16) + 28), dict(dX=(1 << 18) + 16), dict(dX=(1 << 18) - 28),
                                    dict(dX=(1 << 19) + 28), dict(dD=(1 << 17) + 28), dict(dD=(1 << 20) + 4)])
def test_outputs_over_inputs_are_refused(change):
    """k = 8, m = n = 4, batch 2: B and C 32 bytes each, D 32, X, dY and dX 32, dD 32."""
    at = dict(B=1 << 17, C=(1 << 17) + 64, D=1 << 16, X=1 << 18, dY=1 << 19, dX=1 << 20, dD=1 << 21)
    assert grad(**{k: ctypes.c_void_p(v) for k, v in (at | change).items()}) == erm.EINVAL
    assert "overlap" in erm.last_error()
