"""Overlaps of the factored layer's gradient where dX lies in the place of the vectors and another input begins there
too: only those vectors themselves may be where dX is written."""

import ctypes

import pytest

import expanded_rank_matrix_amd as erm

p = ctypes.c_void_p  # never dereferenced: validation fails first
BASE = dict(B=p(1 << 16), C=p(1 << 17), D=p(1 << 18), k=8, m=4, n=6, X=p(1 << 19), dY=p(1 << 20), batch=2, dX=p(1 << 21),
            dD=p(1 << 22), ws=p(1 << 23))


def grad(**change):
    a = {**BASE, **change}
    return erm.load().externd_apply_factors_grad(a["B"], a["C"], a["D"], a["k"], a["m"], a["n"], a["X"], a["dY"], a["batch"],
                                                 a["dX"], a["dD"], a["ws"], None)


@pytest.mark.parametrize("other", ["B", "C", "D", "dY"])
@pytest.mark.parametrize("dD", [BASE["dD"], None])
def test_an_input_that_begins_where_the_vectors_do_is_refused(other, dD):
    assert grad(dX=BASE["X"], dD=dD, **{other: BASE["X"]}) == erm.EINVAL and "overlap" in erm.last_error()


@pytest.mark.parametrize("other", ["B", "C", "D"])
def test_an_input_that_begins_where_dY_does_is_refused(other):
    assert grad(n=4, dX=BASE["dY"], **{other: BASE["dY"]}) == erm.EINVAL and "overlap" in erm.last_error()
