"""The bias's gradient over many pixels: its error does not grow with their number.

Tolerance. A converting thread adds at most 16 chunks in fp32, each the sum of four values: a value passes through at
most 2 + 16 additions, off by half a unit, 2^-24, each. From there the thread's sums are fp64, rounded to fp32 once.
A CTA's threads are added in runs of at most 16 pairs, then eight runs in three steps (1 + 16 + 3), the CTAs in 16 runs
of at most 10, then the runs (10 + 15): 64 * 2^-24 = 2^-18 of the sum of the magnitudes in all, however many pixels
there are."""
import pytest
import torch

import deformable_convolution_sparse_b200 as dcn
from oracle import weight as ow

pytestmark = pytest.mark.gpu

CASES = [
    # M, C, G, K, dtype: the one-pass kernel with one chunk of slots and with two, and the others; rows that TMA takes
    # and rows that it does not
    (27_000_001, 8, 4, 1, torch.bfloat16), (12_000_007, 16, 10, 2, torch.bfloat16),
    (12_000_007, 16, 10, 2, torch.float16), (24_000_003, 8, 4, 1, torch.float32), (24_000_003, 8, 1, 1, torch.bfloat16),
    (8_000_000, 80, 4, 1, torch.bfloat16),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)).replace("torch.", ""))
def test_grad_bias_over_many_pixels(case, cuda_device):
    M, C, G, K, dtype = case
    P = K * K
    NO = 3 * G * P
    y = torch.zeros(M, C, dtype=dtype, device=cuda_device)
    w = torch.zeros(NO, C, dtype=dtype, device=cuda_device)
    # equal values round the same way every time: the longest drift that a running sum can have
    g = (0.1 * (1 + torch.arange(NO, device=cuda_device) / 7)).float().view(1, G, 3 * P).expand(M, -1, -1).contiguous()
    _, gw, gb = dcn.predictor_backward(y, w, g, G=G, K=K)
    assert dcn.device_status() == 0
    sl = torch.tensor(ow.slots(G, P), device=cuda_device)
    want = M * g.double()[0].view(-1)[sl]
    err = (gb.double() - want).abs()
    assert bool((err <= 2.0 ** -18 * want.abs()).all()), float((err / want).max())
    assert not gw.any()
