"""Which tiles the cross entropy's products take, read off the workspace's size: padded rows and the tiles' shares of
the statistics have their place there."""

import ctypes

import pytest

import expanded_rank_matrix_amd as erm

F32, F16, BF16 = 0, 1, 2
SHAPES = [(64, 32), (128, 32), (128, 64), (128, 128), (256, 256)]  # words (or elements of a hidden row) by tokens


def up(a, b):
    return -(-a // b)


def tiles(t, rows, n, vocab):
    """The tile shapes (words, tokens) that the two workspaces' sizes allow."""
    es = 4 if t == F32 else 2
    size = lambda loss: erm.load().externd_token_workspace(t, rows, n, vocab, ctypes.c_void_p(1 << 20), n, loss, 0, 0)  # noqa: E731
    al = lambda b: up(b, 256) * 256  # noqa: E731
    found = []
    for bm, bn in SHAPES:
        padded = up(rows, bn) * bn
        plain = al(8) + al(4 * padded) + al(4 * rows) + al(16 * padded) + al(padded * n * es)
        if size(0) == plain and size(1) == plain + al(4 * padded) + al(up(vocab, bm) * padded * 8):
            found.append((bm, bn))
    assert found, "no shape has this workspace"
    return found


@pytest.mark.parametrize("t,rows,n,vocab", [
    (F32, (1 << 20) - 255, 8256, 1000), (F32, (1 << 20) - 255, 8256, 32000), (F32, (1 << 16) + 1, 1 << 17, 65),
    (F32, (1 << 20) - 255, 1 << 17, 65), (F32, (1 << 20) - 255, 1 << 17, 129), (F32, (1 << 20) - 255, 1 << 17, (1 << 24) - 255),
    (F32, 1, 1 << 17, (1 << 24) - 255), (BF16, (1 << 20) - 255, 1 << 17, 65), (BF16, (1 << 20) - 255, 1 << 16, 65),
    (F16, (1 << 20) - 255, 1 << 17, (1 << 24) - 255), (F16, 1, 1 << 17, 65)])
def test_every_product_fits_a_launch(t, rows, n, vocab):
    """dX's tiles, elements of a hidden row by tokens, with their threads: below 2^32."""
    for bm, bn in tiles(t, rows, n, vocab):
        threads = 128 if bm == 64 else 512 if bm == 256 else 256
        assert up(n, bm) * up(rows, bn) * threads < 1 << 32


@pytest.mark.parametrize("t,rows,vocab,shape", [
    (F32, 65, 10007, (64, 32)), (F32, 257, 32768, (128, 64)), (F32, 600, 32768, (128, 128)), (F32, 1025, 50021, (128, 64)),
    (BF16, 32, 32768, (128, 32)), (BF16, 33, 32768, (128, 64)), (BF16, 65, 32768, (128, 128)), (F16, 300, 50021, (128, 128)),
    (BF16, 2049, 32768, (256, 256))])
def test_every_shape_serves_some_size(t, rows, vocab, shape):
    assert shape in tiles(t, rows, 2560, vocab)
