"""Where the 4-bit products need their workspace: with rows of codes up to 2^22 words apart."""

import pytest

import expanded_rank_matrix_amd as erm

from .test_grouped_cpu import BF16, F16, F32, far, product


@pytest.mark.parametrize("change, word", [(dict(ldq=1 << 22), "workspace"), (dict(ldq=(1 << 22) + 1), "overlap"),
                                          (dict(ldq=(1 << 22) + 1, tokens=64), "overlap"), (dict(ldq=8, tokens=64), "overlap")])
def test_rows_of_codes_far_apart_need_no_workspace(change, word):
    """The output lies over the tokens, which is found after a workspace that is missing."""
    assert product(**{**dict(tokens=100, xt=BF16, ws=None, Y=far[3]), **change}) == erm.EINVAL and word in erm.last_error()


@pytest.mark.parametrize("t,most", [(F32, 32), (F16, 64), (BF16, 64)])
def test_few_tokens_need_no_workspace(t, most):
    size = erm.load().externd_apply_grouped_workspace
    for n, m in ((40, 4), (2560, 2560), (9728, 2560)):
        assert size(t, most, n, m, 32) == 0 and size(t, most + 1, n, m, 32) > 0
