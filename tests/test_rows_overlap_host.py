"""Which arrays of a call the row operators take to share memory, against the bytes
themselves: by the temp query of the embedding gradient, which checks every argument
and enqueues nothing (no GPU)."""
from __future__ import annotations

import numpy as np
import pytest

import sorting_lsd_radix_sort_amd as lrs

A, FAR = 1 << 40, 1 << 42  # fake device addresses, never dereferenced


def refused(grad_y=FAR, ld_gy=64, n=1, ids=2 * FAR, grad=4 * FAR, ld_grad=64, num_ids=1, cols=64):
    try:
        lrs.lrs_embedding_grad(None, 0, "bf16", grad_y, ld_gy, "i64", ids, n, 0, 1.0, "bf16", grad, ld_grad, num_ids,
                               cols, 0, 0)
    except lrs.LrsError as e:
        assert e.status == lrs.LRS_ERR_INVALID_ARG
        return True
    return False


def test_one_row_between_the_rows_of_another_matrix():
    """Halves of one buffer's columns, of which one has a single row (a decode step's
    token beside the rows of its experts): its stride is the buffer's, or not given."""
    for ld in (128, 64, 1):
        for row in (0, 3, 48):
            other = dict(grad=A, ld_grad=128, num_ids=50)
            assert not refused(grad_y=A + 128 + 256 * row, ld_gy=ld, n=1, **other)
            assert refused(grad_y=A + 126 + 256 * row, ld_gy=ld, n=1, **other)
            assert refused(grad_y=A + 130 + 256 * row, ld_gy=ld, n=1, **other)
            # the other way round
            other = dict(grad_y=A, ld_gy=128, n=50)
            assert not refused(grad=A + 128 + 256 * row, ld_grad=ld, num_ids=1, **other)
            assert refused(grad=A + 126 + 256 * row, ld_grad=ld, num_ids=1, **other)
    # ids (8 bytes each) in the columns beside the gradient's, and reaching over into them
    assert not refused(ids=A + 128, n=16, grad=A, ld_grad=128, num_ids=50)
    assert refused(ids=A + 128, n=17, grad=A, ld_grad=128, num_ids=50)
    assert refused(ids=A - 8, n=2, grad=A, ld_grad=128, num_ids=50)


def test_overlap_is_what_the_bytes_say():
    """Matrices of equal stride, or one of a single row, at many distances."""
    rng = np.random.default_rng(1)
    seen = {True: 0, False: 0}
    for _ in range(4000):
        cols = int(rng.integers(1, 6))
        step = int(rng.integers(cols, 3 * cols + 1))
        n, num_ids = (int(v) for v in rng.integers(1, 5, 2))
        gap = int(rng.integers(-step * n - 4, step * num_ids + 4))
        mine = (np.arange(n)[:, None] * step + np.arange(cols)).ravel() + gap
        theirs = (np.arange(num_ids)[:, None] * step + np.arange(cols)).ravel()
        want = bool(np.intersect1d(mine, theirs).size)
        got = refused(grad_y=A + 2 * gap, ld_gy=step, n=n, grad=A, ld_grad=step, num_ids=num_ids, cols=cols)
        assert got == want, (cols, step, n, num_ids, gap)
        seen[want] += 1
    assert min(seen.values()) > 500


@pytest.mark.parametrize("ld", [65, 136])
def test_other_strides_that_meet_are_refused(ld):
    assert refused(grad_y=A, ld_gy=128, n=50, grad=A + 128, ld_grad=ld, num_ids=50)
    assert not refused(grad_y=A, ld_gy=128, n=50, grad=A + 256 * 49 + 128, ld_grad=ld, num_ids=50)
