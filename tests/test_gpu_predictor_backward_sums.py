"""The sums of the predictor's backward: the bias's over many pixels, whose error does not grow with their number, and what
fixes their order.

Tolerance of the bias. A converting thread adds at most 16 chunks in fp32, each the sum of four values: a value passes through at
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


def _shifted(t, shift):
    """A copy of t that starts `shift` elements past a 256-byte boundary."""
    buf = torch.empty(t.numel() + shift, dtype=t.dtype, device=t.device)
    view = buf[shift:].view(t.shape)
    view.copy_(t)
    return view


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16], ids=str)
@pytest.mark.parametrize("M,C,G", [(20000, 64, 4), (3000, 128, 8), (300, 256, 16)])
def test_equal_alignment_gives_equal_bits(M, C, G, dtype, cuda_device):
    """What fixes the sums' order: sizes, dtype and the buffers' 16-byte alignment. Offset views take other kernels
    where TMA cannot read them: the same bits among themselves, and the gradients within their tolerance, (n + 2)
    2^-23 of the sum of the terms' magnitudes, of those of aligned buffers (each within it of the exact sum)."""
    gen = torch.Generator(device=cuda_device).manual_seed(M)
    y = torch.randn(M, C, generator=gen, device=cuda_device).to(dtype)
    w = torch.randn(27 * G, C, generator=gen, device=cuda_device).to(dtype)
    g = torch.randn(M, G, 27, generator=gen, device=cuda_device)
    calls = [dcn.predictor_backward(_shifted(y, s), _shifted(w, s), _shifted(g, s), G=G, K=3) for s in (0, 0, 1, 1)]
    for a, b in (calls[:2], calls[2:]):
        for t, u in zip(a, b):
            assert torch.equal(t, u)
    sl = torch.tensor(ow.slots(G, 9), device=cuda_device)
    gp = g.double().view(M, -1)[:, sl].abs()
    mags = (gp @ w.double().abs(), gp.t() @ y.double().abs(), gp.sum(dim=0))
    for t, u, mag, n in zip(calls[0], calls[2], mags, (27 * G, M, M)):
        assert bool(((t - u).double().abs() <= 2 * (n + 2) * 2.0 ** -23 * mag).all())
