"""Which coefficients dcnv4_orthogonalize takes (no GPU: without its buffers an accepted call stops at the missing
pointers)."""
import pytest

from deformable_convolution_sparse_b200 import binding as B


def _status(a, b, c, steps):
    return B.load_library().dcnv4_orthogonalize(0, 0, 0, 1 << 40, 2, 108, 64, steps, a, b, c, 1e-7, B.DCNV4_F32, None)


@pytest.mark.parametrize("a,b,c,steps", [
    (3.4445, -4.775, 2.0315, 5), (3.4445, -4.775, 2.0315, 64), (1.5, -0.5, 0.0, 64), (1.875, -1.25, 0.375, 64),
    (1.0, 0.0, 0.0, 64), (-1.0, 0.0, 0.0, 3), (3.9, 0.0, 0.0, 1),
    # shrinking as a whole
    (0.5, 0.0, 0.0, 20), (0.5, 0.0, 0.0, 40), (0.5, 0.0, 0.0, 64), (1e-6, 0.0, 0.0, 64), (1e-38, 0.0, 0.0, 64),
    (0.0, 0.0, 0.0, 64), (0.9, 0.05, 0.0, 20), (0.5, 0.5, 0.0, 4), (0.25, 3.0, 0.0, 1),
    (0.0, 1.0, 0.0, 0),
])
def test_taken(a, b, c, steps):
    assert _status(a, b, c, steps) == B.STATUS["DCNV4_ERR_NULL"]


@pytest.mark.parametrize("a,b,c,steps", [
    (4.1, 0.0, 0.0, 1), (1.1, 0.0, 0.0, 20), (100.0, -100.0, 0.0, 1),
    # small singular values fall to less than 1/16 of where the largest can be
    (0.0, 1.0, 0.0, 1), (0.0, 0.0, 1.0, 1), (0.5, 0.5, 0.0, 5), (0.01, 0.0, 0.99, 1), (0.24, 3.76, 0.0, 2),
    (1e-30, 1.0, 0.0, 1),
])
def test_refused(a, b, c, steps):
    assert _status(a, b, c, steps) == B.STATUS["DCNV4_ERR_COEFFICIENTS"]
