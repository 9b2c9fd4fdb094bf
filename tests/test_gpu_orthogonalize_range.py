"""dcnv4_orthogonalize over the whole range of coefficients it takes: iterations that shrink a matrix as well as
ones that let it grow, at the published coefficients and at others, in both of its forms (a matrix per CTA,
a kernel per product), from matrices of any size.

Tolerance of an iteration with b = c = 0, entry by entry: the quotient by the norm is rounded once and the norm is
off by less than that, 2 * 2^-24; in each step P = a I has one entry a row, held to 2^-23, X is held to 2^-23 of
an entry, the products are exact, and their sum, hi hi + hi lo + lo hi, is rounded once and leaves out lo lo, at
most 2^-22 of it: 4.5 * 2^-23 a step, 6 allowed. An entry of X below 2^-16 of what the planes take, 4, is off by
2^-39 of that instead; X's norm lies in [2, 4] in the planes, so that is at most 2^-38 of the norm."""
import numpy as np
import pytest
import torch

import deformable_convolution_sparse_b200 as dcn
from oracle import weight as ow

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


@pytest.mark.parametrize("form", ["", "products"])
@pytest.mark.parametrize("co,steps", [((0.5, 0.0, 0.0), 8), ((0.9, 0.05, 0.0), 12), ((0.6, 0.1, -0.02), 5),
                                      ((1.5, -0.5, 0.0), 12), ((1.875, -1.25, 0.375), 9), ((3.4445, -4.775, 2.0315), 7)],
                         ids=str)
def test_coefficients_of_all_kinds(co, steps, form, cuda_device, monkeypatch):
    """Against the same iteration by fp32 matrix products, both measured against 64 bits: no more than three
    times its error (operands off by 2^-23 where those are off by 2^-24, and truncated additions), plus 2^-22."""
    monkeypatch.setenv("DCNV4_ORTHO_FORM", form)
    for shape in SMALL[1:] + LARGE:
        x = torch.randn(*shape, generator=torch.Generator().manual_seed(sum(shape))).to(cuda_device)
        x[0, 0] *= 1e-3

        def plain(v):
            t = v.shape[1] > v.shape[2]
            v = v.transpose(1, 2) if t else v
            v = v / (torch.linalg.matrix_norm(v, keepdim=True) + 1e-7)
            for _ in range(steps):
                g = v @ v.transpose(1, 2)
                v = co[0] * v + (co[1] * g + co[2] * (g @ g)) @ v
            return v.transpose(1, 2) if t else v
        ref = plain(x.double())
        err = [float((t.double() - ref).norm() / ref.norm())
               for t in (dcn.orthogonalize(x, steps=steps, coefficients=co), plain(x))]
        assert err[0] <= 3 * err[1] + 2.0 ** -22, (shape, err)
    assert dcn.device_status() == 0


@pytest.mark.parametrize("form", ["", "products"])
@pytest.mark.parametrize("scale,eps", [(1e-9, 1.0), (1e-20, 1e-3), (1e-3, 1.0), (1e30, 1e-7), (1e-30, 1e-38)], ids=str)
def test_matrices_of_any_size_keep_their_bits(scale, eps, form, cuda_device, monkeypatch):
    """Norms far below eps, and far from 1, with coefficients that converge (so that a lost plane shows): against
    64 bits, no more than three times the error of fp32 products of the matrix brought to size first."""
    monkeypatch.setenv("DCNV4_ORTHO_FORM", form)
    co, steps = (1.5, -0.5, 0.0), 10
    for shape in ((2, 5, 8), (3, 108, 64), (1, 300, 128)):
        g = torch.Generator().manual_seed(sum(shape))
        x = (torch.randn(*shape, generator=g).double() * scale).float()
        ref = ow.orthogonalize(_np(x), steps, co, float(np.float32(eps)))
        v = torch.tensor(_np(x) / (np.linalg.norm(_np(x), axis=(1, 2), keepdims=True) + float(np.float32(eps))))
        lift = 2.0 ** -np.floor(np.log2(float(v.norm())))
        w, s2 = (v * lift).float().to(cuda_device), lift ** -2.0
        for _ in range(steps):
            w = co[0] * w + s2 * co[1] * (w @ w.transpose(1, 2)) @ w
        out = dcn.orthogonalize(x.to(cuda_device), steps=steps, coefficients=co, eps=eps)
        err = [np.linalg.norm(t - ref) / np.linalg.norm(ref) for t in (_np(out), _np(w) / lift)]
        assert err[0] <= 3 * err[1] + 2.0 ** -22, (shape, err)
    assert dcn.device_status() == 0


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
