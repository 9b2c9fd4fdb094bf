"""Pins of the fp64 definitions of the operators around the predictor's weight
(``oracle.weight``), each against something other than itself."""
import numpy as np
import pytest
import torch

import oracle
from oracle import weight as ow


def test_mx_hand_cases():
    # amax 6 -> floor(log2 6) = 2, scale exponent 0 (byte 127): the elements themselves
    x = np.zeros((1, 32))
    x[0, :12] = [6.0, -4.0, 3.0, 2.0, 1.5, 1.0, 0.5, -0.5, 0.25, 0.75, 2.5, 5.0]
    codes, scales = ow.mx_quantize(x)
    assert scales[0, 0] == 127
    # ties: 0.25 -> 0 and 0.75 -> 1 (even codes 0 and 2), 2.5 -> 2, 5 -> 4
    assert list(codes[0, 0, :12]) == [7, 14, 5, 4, 3, 2, 1, 9, 0, 2, 4, 6]
    # amax 7.9 keeps the exponent of 6: values above 6 saturate
    x = np.zeros((1, 32))
    x[0, 0], x[0, 1] = 7.9, -7.9
    codes, scales = ow.mx_quantize(x)
    assert scales[0, 0] == 127 and list(codes[0, 0, :2]) == [7, 15]
    # amax 8 takes the next one: 8 = 4 * 2
    x[0, 0] = 8.0
    codes, scales = ow.mx_quantize(x)
    assert scales[0, 0] == 128 and codes[0, 0, 0] == 6
    assert ow.mx_values(codes, scales, 2)[0, 0] == 8.0


def test_mx_edges():
    x = np.zeros((5, 33))
    x[1, 32] = 2.0 ** -140      # the scale exponent stops at -127
    x[2, 0] = np.inf
    x[3, 5] = np.nan
    x[4, 0] = 2.0 ** 127
    codes, scales = ow.mx_quantize(x)
    assert scales.tolist() == [[0, 0], [0, 0], [255, 0], [255, 0], [252, 0]]
    assert codes[1, 1, 0] == 0 and codes[4, 0, 0] == 6
    v = ow.mx_values(codes, scales, 33)
    assert np.isnan(v[2, :32]).all() and v[2, 32] == 0.0 and v[4, 0] == 2.0 ** 127


def test_mx_values_are_the_nearest_of_the_grid():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((20, 64)) * np.exp(3 * rng.standard_normal((20, 1)))
    codes, scales = ow.mx_quantize(x)
    v = ow.mx_values(codes, scales, 64)
    grid = np.concatenate([ow.E2M1, -ow.E2M1])
    for m in range(20):
        for c in range(64):
            g = grid * 2.0 ** (int(scales[m, c // 32]) - 127)
            assert abs(v[m, c] - x[m, c]) == np.abs(g - x[m, c]).min()
    assert np.array_equal(ow.mx_unpack(ow.mx_pack(codes)), codes)


@pytest.mark.parametrize("G,P", [(1, 1), (2, 9), (4, 8), (3, 25)])
def test_slots_follow_the_c_oracle(G, P):
    # a projection that gives channel o the value o: its records hold the channel of every slot
    NO = 3 * G * P
    rec = oracle.dcnv4_predictor(np.ones((1, 1)), np.zeros((NO, 1)), np.arange(NO, dtype=float), G=G, P=P).reshape(-1)
    assert np.array_equal(rec[ow.slots(G, P)], np.arange(NO))


def test_predictor_backward_is_the_derivative():
    rng = np.random.default_rng(1)
    G, P, C, M = 2, 4, 7, 5
    y, w = rng.standard_normal((M, C)), rng.standard_normal((3 * G * P, C))
    b, g = rng.standard_normal(3 * G * P), rng.standard_normal((M, G, 3 * P))

    def loss(y, w, b):
        return float((oracle.dcnv4_predictor(y, w, b, G=G, P=P).reshape(g.shape) * g).sum())

    gy, gw, gb = ow.predictor_backward(y, w, g, G, P)
    h = 1e-4   # the loss is linear in each argument: differences are exact up to rounding
    for t, grad in ((y, gy), (w, gw), (b, gb)):
        for i in np.ndindex(*t.shape):
            t[i] += h
            up = loss(y, w, b)
            t[i] -= 2 * h
            dn = loss(y, w, b)
            t[i] += h
            assert abs((up - dn) / (2 * h) - grad[i]) <= 1e-9


@pytest.mark.parametrize("R,C", [(3, 5), (5, 3), (4, 4), (1, 6), (6, 1)])
def test_orthogonalize_moves_the_singular_values_by_the_polynomial(R, C):
    x = np.random.default_rng(R * 10 + C).standard_normal((2, R, C))
    a, b, c = co = (3.4445, -4.7750, 2.0315)
    got = ow.orthogonalize(x, 5, co, 1e-7)
    for i in range(2):
        u, s, vt = np.linalg.svd(x[i] / (np.linalg.norm(x[i]) + 1e-7), full_matrices=False)
        for _ in range(5):
            s = a * s + b * s ** 3 + c * s ** 5
        assert np.abs(u @ np.diag(s) @ vt - got[i]).max() <= 1e-12


def test_orthogonalize_converges_to_the_polar_factor():
    # (15/8, -5/4, 3/8) has a fixed point at 1 of third order
    x = np.random.default_rng(3).standard_normal((1, 6, 9))
    u, _, vt = np.linalg.svd(x[0], full_matrices=False)
    got = ow.orthogonalize(x, 20, (1.875, -1.25, 0.375))
    assert np.abs(got[0] - u @ vt).max() <= 1e-12
    # an independent evaluation in torch
    t = torch.tensor(x[0])
    t = t / (t.norm() + 1e-7)
    for _ in range(20):
        t = 1.875 * t - 1.25 * (t @ t.T @ t) + 0.375 * (t @ t.T @ t @ t.T @ t)
    assert np.abs(t.numpy() - got[0]).max() <= 1e-12
