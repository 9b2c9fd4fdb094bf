"""dcnv4_orthogonalize over the whole range of coefficients it takes: iterations that shrink a matrix as well as
ones that let it grow, in both of its forms (a matrix per CTA, a kernel per product).

Tolerance of an iteration with b = c = 0, entry by entry: the quotient by the norm is rounded once and the norm is
off by less than that, 2 * 2^-24; in each step P = a I has one entry a row, held to 2^-23, X is held to 2^-23 of
an entry, the products are exact, and their sum, hi hi + hi lo + lo hi, is rounded once and leaves out lo lo, at
most 2^-22 of it: 4.5 * 2^-23 a step, 6 allowed. An entry of X below 2^-16 of what the planes take, 4, is off by
2^-39 of that instead; X's norm lies in [2, 4] in the planes, so that is at most 2^-38 of the norm."""
import numpy as np
import pytest
import torch

import deformable_convolution_sparse_b200 as dcn

pytestmark = pytest.mark.gpu

SMALL = [(1, 1, 1), (2, 5, 8), (3, 108, 64), (2, 33, 130), (1, 60, 384)]      # one CTA holds them
LARGE = [(2, 129, 257), (1, 300, 128), (1, 520, 600)]


def _np(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("form", ["", "products"])
@pytest.mark.parametrize("steps", [1, 20, 40, 64])
@pytest.mark.parametrize("a", [0.5, -0.7, 0.001, 1.0, 3.0])
def test_coefficients_that_scale_the_matrix(a, steps, form, cuda_device, monkeypatch):
    """X -> a^steps X / (norm + eps), also when a^steps is far below what 16 bits hold."""
    if abs(a) ** steps > 4 or (abs(a) < 0.01 and steps > 12):
        steps = 1 if a > 1 else 12   # (0.001^12: 1e-36, near the end of fp32)
    monkeypatch.setenv("DCNV4_ORTHO_FORM", form)
    for shape in SMALL + LARGE:
        x = torch.randn(*shape, generator=torch.Generator().manual_seed(sum(shape))) * 0.1
        out = dcn.orthogonalize(x.to(cuda_device), steps=steps, coefficients=(a, 0.0, 0.0))
        assert dcn.device_status() == 0
        af = float(np.float32(a))
        X = _np(x)
        want = af ** steps * X / (np.sqrt((X * X).sum(axis=(1, 2), keepdims=True)) + float(np.float32(1e-7)))
        err = np.abs(_np(out) - want)
        floor = steps * 2.0 ** -38 * np.linalg.norm(want, axis=(1, 2), keepdims=True) + 2.0 ** -149   # (fp32's last)
        assert np.all(err <= (2 + 12 * steps) * 2.0 ** -24 * np.abs(want) + floor), (shape, (err / np.abs(want)).max())


def test_coefficients_that_let_small_singular_values_fall_behind_are_refused(cuda_device):
    x = torch.randn(3, 40, 50, device=cuda_device)
    for co, steps in (((0.0, 1.0, 0.0), 1), ((0.5, 0.5, 0.0), 5), ((0.01, 0.0, 0.99), 1)):
        with pytest.raises(dcn.DCNv4Error, match="COEFFICIENTS"):
            dcn.orthogonalize(x, steps=steps, coefficients=co)


@pytest.mark.parametrize("form", ["", "products"])
def test_coefficients_at_the_end_of_fp32(form, cuda_device, monkeypatch):
    """Zeros give zeros; a step that leaves nothing above fp32's subnormals gives those or zeros, no NaN."""
    monkeypatch.setenv("DCNV4_ORTHO_FORM", form)
    for shape in ((3, 40, 50), (1, 150, 140)):
        x = torch.randn(*shape, device=cuda_device)
        for steps in (1, 5):
            assert not dcn.orthogonalize(x, steps=steps, coefficients=(0.0, 0.0, 0.0)).any()
            for a in (1e-45, 1e-38):
                out = dcn.orthogonalize(x, steps=steps, coefficients=(a, 0.0, 0.0))
                assert torch.isfinite(out).all() and float(out.abs().max()) <= 1.01 * a
        # a matrix of 2^-100 that shrinks: 2^-140, subnormal in fp32
        want = x.double() / (torch.linalg.matrix_norm(x.double(), keepdim=True) * 2.0 ** -100 + 1.0) * 2.0 ** -140
        out = dcn.orthogonalize(x * 2.0 ** -100, steps=4, coefficients=(2.0 ** -10, 0.0, 0.0), eps=1.0)
        assert bool(((out.double() - want).abs() <= 2.0 ** -148).all())
