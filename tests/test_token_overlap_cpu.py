"""Overlaps of the token loss's arguments where a gradient lies in the place of X and another input begins there too:
only X itself may be where dX is written."""

import pytest

import expanded_rank_matrix_amd as erm

from .test_token_cpu import BASE, grad, loss, p

X = BASE["X"]


@pytest.mark.parametrize("change", [
    dict(W=X), dict(W=X, dW=None), dict(W=X, vocab=1, dW=None), dict(target=X), dict(weight=X),
    dict(W=X, ldx=16, lddx=16, ldw=16)])
def test_another_input_that_begins_where_x_does_is_refused(change):
    for entry in (loss, grad):
        assert entry(**{**BASE, "dX": X, **change}) == erm.EINVAL and "overlap" in erm.last_error()


def test_statistics_that_begin_where_x_does_are_refused():
    assert grad(dX=X, stats=X) == erm.EINVAL and "overlap" in erm.last_error()


def test_dW_in_the_place_of_both_is_refused():
    for entry in (loss, grad):
        assert entry(dX=X, dW=X) == erm.EINVAL and "overlap" in erm.last_error()
