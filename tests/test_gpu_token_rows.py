"""The token loss at sizes of many rows: each shape of tiles that fp32 takes, against the definition in 64 bits, with the
tolerances that are derived beside it."""

import pytest
import torch

from .test_gpu_token import check, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,vocab", [(65, 10007), (300, 32768), (600, 32768), (1024, 32700)])
@pytest.mark.parametrize("n", [68, 61])
def test_fp32_in_tiles_of_every_shape(rows, vocab, n):
    x, w, target, weight = inputs(rows, n, vocab, torch.float32)
    target[1::9] = -100
    check(x, w, target, weight)
