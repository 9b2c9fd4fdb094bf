"""The paths of orthogonalize that other tests run with the Muon coefficients alone, with coefficients that converge
(1.5, -0.5, 0 and 1.875, -1.25, 0.375): those pass errors on without blowing them up, so that the bound on the error,
a step's rounding of 8 * 2^-22 of its terms carried through the following steps' largest derivatives, is tight enough
to show a lost plane (operands of 11 bits are 6 to 38 times over it)."""
import numpy as np
import pytest
import torch

import deformable_convolution_sparse_b200 as dcn

pytestmark = pytest.mark.gpu

COEFFICIENTS = [(1.5, -0.5, 0.0), (1.875, -1.25, 0.375)]


def _np(t):
    return t.detach().double().cpu().numpy()


def _reference(x, steps, co, eps):
    """(fp64 result, Frobenius tolerance in fp32) per matrix."""
    a, b, c = co
    for X in _np(x):
        X = X / (np.linalg.norm(X) + eps)
        local, growth, r = [2.0 ** -22 * np.linalg.norm(X)], [], 1.0
        for _ in range(steps):
            local.append(8 * 2.0 ** -22 * (abs(a) + abs(b) * r ** 2 + abs(c) * r ** 4) * np.linalg.norm(X))
            s = np.linspace(0, r, 2001)
            growth.append(np.abs(a + 3 * b * s ** 2 + 5 * c * s ** 4).max())
            r = np.abs(a * s + b * s ** 3 + c * s ** 5).max()
            A = X @ X.T
            X = a * X + (b * A + c * (A @ A)) @ X
        total, g = 0.0, 1.0
        for k in range(steps, -1, -1):
            total += local[k] * g
            if k:
                g *= growth[k - 1]
        yield X, total + 2.0 ** -24 * np.linalg.norm(X)


def _check(out, x, steps, co, eps=1e-7):
    for got, (ref, tol) in zip(_np(out), _reference(x, steps, co, eps)):
        err = np.linalg.norm(got - ref)
        assert err <= tol, (x.shape, err, tol)


@pytest.mark.parametrize("form", ["", "products"])
@pytest.mark.parametrize("co", COEFFICIENTS, ids=str)
@pytest.mark.parametrize("shape", [(2, 5, 8), (3, 108, 64), (2, 129, 257), (1, 300, 128), (1, 60, 384), (1, 64, 385),
                                   (20, 256, 200), (1, 900, 700)], ids=lambda c: "x".join(map(str, c)))
def test_both_forms(shape, co, form, cuda_device, monkeypatch):
    """One CTA a matrix, a kernel per product with more tiles than SMs and with fewer, with long sums and short."""
    monkeypatch.setenv("DCNV4_ORTHO_FORM", form)
    x = torch.randn(*shape, generator=torch.Generator().manual_seed(sum(shape)))
    out = dcn.orthogonalize(x.to(cuda_device), coefficients=co)
    assert dcn.device_status() == 0
    _check(out, x, 5, co)


@pytest.mark.parametrize("co", COEFFICIENTS, ids=str)
@pytest.mark.parametrize("shape", [(6, 16, 24), (6, 150, 140)], ids=["small", "tiles"])
def test_extreme_matrices(shape, co, cuda_device):
    g = torch.Generator().manual_seed(0)
    x = torch.randn(*shape, generator=g)
    x[1] = 0.0
    x[2, 3, 5] = float("nan")
    x[3, 0, 0] = float("inf")
    x[4] *= 1e30
    x[5] *= 1e-30
    out = dcn.orthogonalize(x.to(cuda_device), coefficients=co, eps=1e-38)
    assert not out[1].any() and torch.isnan(out[2]).all() and torch.isnan(out[3]).all()
    _check(out[[0, 4, 5]], x[[0, 4, 5]], 5, co, float(np.float32(1e-38)))
    for scale, eps in ((1e-9, 1.0), (1e-3, 1.0), (1e-25, 1e-20)):   # norms far below eps: lifted on the way
        tiny = torch.randn(1, *shape[1:], generator=g) * scale
        _check(dcn.orthogonalize(tiny.to(cuda_device), coefficients=co, eps=eps), tiny, 5, co, float(np.float32(eps)))


@pytest.mark.parametrize("co", COEFFICIENTS, ids=str)
def test_low_rank_and_a_weight_gradient(co, cuda_device):
    g = torch.Generator().manual_seed(6)
    x = torch.matmul(torch.randn(2, 64, 3, generator=g), torch.randn(2, 3, 96, generator=g))
    _check(dcn.orthogonalize(x.to(cuda_device), coefficients=co), x, 5, co)
    y = torch.randn(3000, 64, generator=g).half().to(cuda_device)
    w = (torch.randn(108, 64, generator=g) / 8).half().to(cuda_device)
    gr = torch.randn(3000, 4, 27, generator=g).to(cuda_device)
    gw = dcn.predictor_backward(y, w, gr, G=4, K=3)[1]
    _check(dcn.orthogonalize(gw, coefficients=co)[None], gw[None], 5, co)
