"""fp64 definitions of the operators around the predictor's weight.

TEST INFRASTRUCTURE ONLY, as the package's C oracle: plain numpy in fp64,
sharing no code with the CUDA path. Pinned by
``tests/test_oracle_weight_pins.py``.

Microscaled 4-bit format: the OCP Microscaling Formats specification v1.0
(MXFP4), scale exponent floor(log2(amax)) - 2 held to [-127, ...], elements
rounded to nearest, ties to even, saturating. A block with a non-finite value
is a block of NaN. Projection and records: as ``oracle.dcnv4_predictor``.
Newton-Schulz: X / (|X|_F + eps), then X <- aX + (bA + cAA)X with A = XX^T.
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = 32


def mx_quantize(x: np.ndarray):
    """(element codes 0..15 [M, nb, 32], scale bytes [M, nb]) of x [M, C]."""
    x = np.asarray(x, dtype=np.float64)
    M, C = x.shape
    nb = -(-C // BLOCK)
    v = np.zeros((M, nb * BLOCK))
    v[:, :C] = x
    v = v.reshape(M, nb, BLOCK)
    codes = np.zeros(v.shape, dtype=np.uint8)
    scales = np.zeros((M, nb), dtype=np.uint8)
    for m in range(M):
        for b in range(nb):
            blk = v[m, b]
            if not np.all(np.isfinite(blk)):
                scales[m, b] = 255
                continue
            amax = np.max(np.abs(blk)) if BLOCK else 0.0
            # frexp: amax = f * 2^k with f in [1/2, 1), so floor(log2(amax)) = k - 1
            e = -127 if amax == 0.0 else max(int(np.frexp(amax)[1]) - 1 - 2, -127)
            scales[m, b] = e + 127
            q = np.ldexp(np.abs(blk), -e)
            # nearest of the 8 magnitudes; of two equally near ones the even code
            d = np.abs(q[:, None] - E2M1[None, :])
            near = d == d.min(axis=1, keepdims=True)
            code = np.where(near.sum(axis=1) == 2,
                            np.where(near[:, ::2].any(axis=1), 2 * near[:, ::2].argmax(axis=1), 0),
                            near.argmax(axis=1))
            codes[m, b] = code.astype(np.uint8) | (np.signbit(blk).astype(np.uint8) << 3)
    return codes, scales


def mx_pack(codes: np.ndarray) -> np.ndarray:
    """Bytes [M, nb * 16]: element 2i of a block in the low half of byte i, 2i + 1 in the high half."""
    M = codes.shape[0]
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).reshape(M, -1)


def mx_unpack(packed: np.ndarray) -> np.ndarray:
    M, n = packed.shape
    codes = np.empty((M, 2 * n), dtype=np.uint8)
    codes[:, 0::2], codes[:, 1::2] = packed & 15, packed >> 4
    return codes.reshape(M, n // 16, BLOCK)


def mx_values(codes: np.ndarray, scales: np.ndarray, C: int) -> np.ndarray:
    """fp64 values [M, C]."""
    v = E2M1[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    e = scales.astype(np.int64) - 127
    v = np.ldexp(v, e[..., None].astype(np.int32))
    v = np.where((scales == 255)[..., None], np.nan, v)
    return v.reshape(codes.shape[0], -1)[:, :C]


def slots(G: int, P: int) -> np.ndarray:
    """Record slot of every projection channel, by moving the channel numbers through the records' reshape."""
    o = np.arange(3 * G * P)
    rec = np.concatenate([o[:2 * G * P].reshape(G, 2 * P), o[2 * G * P:].reshape(G, P)], axis=1).reshape(-1)
    s = np.empty(3 * G * P, dtype=np.int64)
    s[rec] = np.arange(3 * G * P)
    return s


def predictor_backward(y, weight, grad_records, G: int, P: int):
    """(grad_y [M, C], grad_weight [3GP, C], grad_bias [3GP]) for grad_records [M, G, 3P]."""
    y, weight = np.asarray(y, np.float64), np.asarray(weight, np.float64)
    gp = np.asarray(grad_records, np.float64).reshape(-1, 3 * G * P)[:, slots(G, P)]
    return gp @ weight, gp.T @ y, gp.sum(axis=0)


def orthogonalize(x, steps: int = 5, coefficients=(3.4445, -4.7750, 2.0315), eps: float = 1e-7) -> np.ndarray:
    """x [B, R, C]."""
    a, b, c = coefficients
    out = np.array(x, dtype=np.float64)
    for i in range(out.shape[0]):
        X = out[i]
        X = X / (np.sqrt(np.sum(X * X)) + eps)
        for _ in range(steps):
            A = X @ X.T
            X = a * X + (b * A + c * (A @ A)) @ X
        out[i] = X
    return out
