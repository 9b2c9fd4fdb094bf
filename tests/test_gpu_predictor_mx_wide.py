"""predictor_mx on as many pixels as large batches have: more tiles than SMs, so that a CTA takes as many record slots
as it can hold (a few pixels take tiles of 16 or 32 slots): two groups of weight scales, several swizzled column
blocks a tile, several wide slot tiles. Against the fp64 definition on a sample of rows: whole tiles at the start, in
the middle and at the end, and scattered ones.

Tolerance: a sum of C exact products in fp32, in any order and with truncated additions, is off by at most
(C + 2) 2^-23 sum|terms|; the output adds half a unit of its type."""
import numpy as np
import pytest
import torch

import oracle
import deformable_convolution_sparse_b200 as dcn
from oracle import weight as ow

pytestmark = pytest.mark.gpu

TD = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TINY = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}   # half the spacing of the subnormals

CASES = [
    # M, C, G, K, remove_center, bias
    (20001, 256, 16, 3, False, True),   # 432 slots in two tiles
    (20000, 320, 8, 3, True, True),     # 192 slots, ten blocks of channels
    (20011, 160, 8, 3, False, False),   # 216 slots, an odd number of blocks
    (19999, 512, 32, 3, False, True),   # 864 slots in four tiles
    (40001, 64, 8, 3, False, True),     # 216 slots, two blocks
    (20005, 100, 7, 3, False, True),    # 189 slots: rows that TMA does not take; channels that end inside a block
    (30003, 300, 4, 4, False, True),    # 192 slots
]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
def test_predictor_mx_over_many_tiles(case, dtype, cuda_device):
    M, C, G, K, rc, bias = case
    P = K * K - (1 if rc else 0)
    NO = 3 * G * P
    gen = torch.Generator().manual_seed(M + C)
    y = torch.randn(M, C, generator=gen) * torch.exp(torch.randn(C, generator=gen))
    y[::11] = 0.0
    y = y.to(TD[dtype])
    w = torch.randn(NO, C, generator=gen) * C ** -0.5 * torch.exp(torch.randn(NO, 1, generator=gen))
    wq = ow.mx_quantize(w.double().numpy())
    b = torch.randn(NO, generator=gen) if bias else None
    out = dcn.predictor_mx(y.to(cuda_device), torch.tensor(ow.mx_pack(wq[0])).to(cuda_device),
                           torch.tensor(wq[1]).to(cuda_device), None if b is None else b.to(cuda_device), G=G, K=K,
                           remove_center=rc)
    assert dcn.device_status() == 0
    mid = M // 256 * 128
    rows = torch.unique(torch.cat([torch.arange(128), torch.arange(mid, mid + 128), torch.arange(M - 160, M),
                                   torch.randint(M, (64,), generator=gen)]))
    q = ow.mx_values(*ow.mx_quantize(y[rows].double().numpy()), C)
    wv, bv = ow.mx_values(*wq, C), None if b is None else b.double().numpy()
    ref = oracle.dcnv4_predictor(q, wv, bv, G=G, P=P).reshape(len(rows), -1)
    mag = oracle.dcnv4_predictor(np.abs(q), np.abs(wv), None if bv is None else np.abs(bv), G=G, P=P).reshape(len(rows), -1)
    err = np.abs(out[rows.to(cuda_device)].double().cpu().numpy().reshape(ref.shape) - ref)
    tol = torch.finfo(TD[dtype]).eps / 2 * np.abs(ref) * (1 + 2.0 ** -10) + TINY[dtype] + (C + 2) * 2.0 ** -23 * mag
    at = np.unravel_index(np.argmax(err - tol), err.shape)
    assert np.all(err <= tol), f"{(err - tol).max():.3e} over at pixel {int(rows[at[0]])}, slot {at[1]}"
    # the other rows: the same bits as in a call of their own, whose tiles hold other pixels
    part = slice(M // 3, M // 3 + 19000)
    again = dcn.predictor_mx(y[part].to(cuda_device), torch.tensor(ow.mx_pack(wq[0])).to(cuda_device),
                             torch.tensor(wq[1]).to(cuda_device), None if b is None else b.to(cuda_device), G=G, K=K,
                             remove_center=rc)
    assert torch.equal(again, out[part])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("ly,lw", [(-126, 0), (-126, -3), (-60, -66), (-126, 120), (120, -126), (126, 0), (-100, -40)])
def test_predictor_mx_at_the_ends_of_the_scales(ly, lw, dtype, cuda_device):
    """Activations of 2^ly and weights of 2^lw: sums down to fp32's subnormals and up to its largest number. (Each sum
    is off by up to a unit of the subnormals, 2^-149, too.)"""
    M, C, G = 300, 96, 2
    gen = torch.Generator().manual_seed(ly + lw)
    y = (torch.randn(M, C, generator=gen) * 0.3 * 2.0 ** ly).to(TD[dtype])
    w = torch.randn(54, C, generator=gen) * 0.3 * 2.0 ** lw
    codes, scales = dcn.mx_quantize(w.to(cuda_device))
    out = dcn.predictor_mx(y.to(cuda_device), codes, scales, None, G=G, K=3)
    q = ow.mx_values(*ow.mx_quantize(y.double().numpy()), C)
    wv = ow.mx_values(ow.mx_unpack(codes.cpu().numpy()), scales.cpu().numpy(), C)
    ref = oracle.dcnv4_predictor(q, wv, None, G=G, P=9).reshape(M, -1)
    mag = oracle.dcnv4_predictor(np.abs(q), np.abs(wv), None, G=G, P=9).reshape(M, -1)
    got = out.double().cpu().numpy().reshape(M, -1)
    assert not np.isnan(got).any()
    tol = torch.finfo(TD[dtype]).eps / 2 * np.abs(ref) * (1 + 2.0 ** -10) + TINY[dtype] + (C + 2) * 2.0 ** -23 * mag + 2.0 ** -149
    inside = np.abs(ref) + tol < torch.finfo(TD[dtype]).max
    assert np.all((np.abs(got - ref) <= tol)[inside])
    assert np.all(np.abs(got[np.abs(ref) > 3.5e38]) > 3.3e38)   # past the end: infinite, or the largest number
