"""GPU parity of the operators around the predictor's weight (4-bit microscaled
quantisation and projection, the predictor's backward, the orthogonalised
update) against their fp64 definitions, at the sizes and values where they can
go wrong, and as they are used together.

Tolerances. Quantisation is exact: codes and scales are compared as integers,
values read back as the exact value rounded once. A sum of n fp32 terms, in any
order and with truncated additions, is off by at most (n + 2) 2^-23 sum|terms|
(each addition and each product at most a whole unit 2^-23 of a partial sum);
an output in T adds half a unit of T. The orthogonalised update is bounded
in the Frobenius norm: a step's rounding, 8 * 2^-22 of the size of its terms
(operands of 22 bits, errors of the many terms independent, a factor 8 for the
spread), then grows by at most max|phi'| per following step, phi(s) =
a s + b s^3 + c s^5 (the derivative of an odd matrix function is bounded by
that of its scalar function).
"""
import numpy as np
import pytest
import torch

import oracle
import deformable_convolution_sparse_b200 as dcn
from deformable_convolution_sparse_b200 import binding
from oracle import weight as ow

pytestmark = pytest.mark.gpu

TD = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_UNIT = {k: torch.finfo(t).eps / 2 for k, t in TD.items()}
TINY = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}   # half the spacing of the subnormals
U = 2.0 ** -23


def _np(t):
    return t.detach().double().cpu().numpy()


def _guarded(shape, dtype, dev, shift=0, fill=7.0):
    """A tensor inside a larger buffer of known contents, `shift` elements off its alignment."""
    n, guard = int(np.prod(shape)), 64
    buf = torch.full((n + 2 * guard + shift,), fill, dtype=dtype, device=dev)
    view = buf[guard + shift:guard + shift + n].view(shape)

    def untouched():
        return bool(torch.all(buf[:guard + shift] == fill)) and bool(torch.all(buf[guard + shift + n:] == fill))
    return view, untouched


# -------------------------------------------------------------- quantisation ---

def _mx_input(M, C, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, C, generator=g) * torch.exp(2 * torch.randn(M, 1, generator=g))
    x[::7] = 0.0
    if M > 8 and C > 2:
        # exact ties and range ends of the grid, signed zeros, the ends of the storage type
        t = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -5.0, 6.0, 7.9, -0.0, 4.0, 0.5])
        x[1, :min(C, 14)] = t[:min(C, 14)]
        if C >= 14:
            x[1, 9] = 4.5   # keeps the block's exponent
        x[2, 0], x[3, 0] = float("inf"), float("nan")
        fi = torch.finfo(TD[dtype])
        x[4, 0], x[5, 0], x[5, 1] = fi.max, fi.tiny, fi.tiny * fi.eps
        x[6] = fi.tiny * fi.eps
        x[8, :] = -0.0
    return x.to(TD[dtype])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,C", [(1, 1), (3, 31), (40, 32), (17, 33), (130, 64), (9, 77), (11, 320), (1000, 24)])
def test_mx_quantize_and_back(M, C, dtype, cuda_device):
    x = _mx_input(M, C, dtype, seed=M + C)
    rc, rs = ow.mx_quantize(_np(x))
    for shift in (0, 1):   # 1: rows not 16-byte aligned
        xd, _ = _guarded((M, C), TD[dtype], cuda_device, shift)
        xd.copy_(x)
        codes, scales = dcn.mx_quantize(xd)
        assert np.array_equal(scales.cpu().numpy(), rs)
        assert np.array_equal(ow.mx_unpack(codes.cpu().numpy()), rc)
        for back in ("f32", "f16", "bf16"):
            out, untouched = _guarded((M, C), TD[back], cuda_device, shift)
            assert dcn.mx_dequantize(codes, scales, C, TD[back], out=out) is out
            want = torch.tensor(ow.mx_values(rc, rs, C)).to(TD[back])   # fp64 rounded once
            assert torch.equal(torch.nan_to_num(out.cpu(), nan=123.0), torch.nan_to_num(want, nan=123.0))
            assert untouched()


def test_mx_quantize_outputs_stay_in_their_bounds_and_take_leading_shapes(cuda_device):
    x = torch.randn(3, 5, 2, 70, device=cuda_device)
    codes, uc = _guarded((3, 5, 2, 48), torch.uint8, cuda_device, shift=0, fill=7)
    scales, us = _guarded((3, 5, 2, 3), torch.uint8, cuda_device, shift=1, fill=7)
    dcn.mx_quantize(x, codes, scales)
    assert uc() and us()
    rc, rs = ow.mx_quantize(_np(x).reshape(30, 70))
    assert np.array_equal(ow.mx_unpack(codes.cpu().numpy().reshape(30, 48)), rc)
    assert np.array_equal(scales.cpu().numpy().reshape(30, 3), rs)
    assert dcn.mx_quantize(x[:0])[0].shape == (0, 5, 2, 48)
    assert dcn.mx_dequantize(codes[:0], scales[:0], 70).shape == (0, 5, 2, 70)
    with pytest.raises(ValueError):
        dcn.mx_dequantize(codes, scales, 97)
    with pytest.raises(ValueError):
        dcn.mx_quantize(x.transpose(0, 1))


# ---------------------------------------------------------- 4-bit projection ---

def _mx_weight(NO, C, seed, dev):
    g = torch.Generator().manual_seed(seed)
    w = torch.randn(NO, C, generator=g) * C ** -0.5 * torch.exp(torch.randn(NO, 1, generator=g))
    w[0] = 0.0
    codes, scales = ow.mx_quantize(w.double().numpy())
    return (torch.tensor(ow.mx_pack(codes)).to(dev), torch.tensor(scales).to(dev), ow.mx_values(codes, scales, C))


def _check_mx_projection(got, y, wv, b, G, P, dtype):
    q = ow.mx_values(*ow.mx_quantize(_np(y)), y.shape[1])
    ref = oracle.dcnv4_predictor(q, wv, b, G=G, P=P).reshape(-1, 3 * G * P)
    mag = oracle.dcnv4_predictor(np.abs(q), np.abs(wv), None if b is None else np.abs(b), G=G, P=P).reshape(-1, 3 * G * P)
    err = np.abs(_np(got).reshape(ref.shape) - ref)
    tol = HALF_UNIT[dtype] * np.abs(ref) * (1 + 2.0 ** -10) + TINY[dtype] + (y.shape[1] + 2) * U * mag
    assert np.all(err <= tol), f"{np.max(err - tol):.3e} over, at {np.unravel_index(np.argmax(err - tol), err.shape)}"


MX_CASES = [
    # M, C, G, K, remove_center, bias
    (1, 64, 4, 3, False, True),        # one pixel
    (129, 64, 4, 3, False, False),     # one pixel over a tile
    (1000, 128, 8, 3, False, True),    # 216 channels
    (300, 256, 16, 3, False, True),    # 432 channels: the stage-3 projection
    (77, 320, 8, 3, True, True),       # no centre: 192 channels, 5 x 64 input channels
    (260, 512, 32, 3, False, True),    # 864 channels
    (65, 32, 1, 1, False, True),       # three channels
    (140, 8, 2, 5, False, True),       # C below a block
    (200, 33, 3, 3, False, True),      # one channel in the last block, odd rows
    (131, 100, 5, 3, False, False),    # 135 channels
    (90, 1056, 2, 3, False, True),     # 33 blocks
    (500, 96, 8, 3, False, True),      # 3 blocks, 512-thread CTAs: the last round of pieces is half empty
    (300, 72, 8, 3, False, False),     # the same, a quarter of the last block
    (1300, 160, 8, 3, False, True),
    (40, 4000, 1, 1, False, True),     # rows too long for the tensor-core kernel
    (20000, 64, 4, 3, False, True),    # several tiles per SM
]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", MX_CASES, ids=lambda c: "x".join(map(str, c)))
def test_predictor_mx(case, dtype, cuda_device):
    M, C, G, K, rc, bias = case
    P = K * K - (1 if rc else 0)
    NO = 3 * G * P
    g = torch.Generator().manual_seed(M + C)
    y = torch.randn(M, C, generator=g) * torch.exp(torch.randn(C, generator=g))
    y[::11] = 0.0
    y = y.to(TD[dtype])
    codes, scales, wv = _mx_weight(NO, C, M, cuda_device)
    b = torch.randn(NO, generator=g) if bias else None
    out, untouched = _guarded((M, G, 3 * P), TD[dtype], cuda_device)
    dcn.predictor_mx(y.to(cuda_device), codes, scales, None if b is None else b.to(cuda_device), G=G, K=K,
                     remove_center=rc, out=out)
    assert dcn.device_status() == 0
    assert untouched()
    _check_mx_projection(out, y, wv, None if b is None else b.double().numpy(), G, P, dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_predictor_mx_misaligned_rows_and_nan_pixels(dtype, cuda_device):
    M, C, G, K = 200, 64, 2, 3
    codes, scales, wv = _mx_weight(54, C, 1, cuda_device)
    y, _ = _guarded((M, C), TD[dtype], cuda_device, shift=1)
    y.copy_(torch.randn(M, C, generator=torch.Generator().manual_seed(1)))
    out, untouched = _guarded((M, G, 27), TD[dtype], cuda_device, shift=1)
    dcn.predictor_mx(y, codes, scales, None, G=G, K=K, out=out)
    assert untouched()
    _check_mx_projection(out, y.cpu(), wv, None, G, 9, dtype)
    clean = out.clone()
    y[3, 5], y[150, 63] = float("nan"), float("-inf")
    dcn.predictor_mx(y, codes, scales, None, G=G, K=K, out=out)
    bad = torch.zeros(M, dtype=torch.bool, device=cuda_device)
    bad[3] = bad[150] = True
    # weights of zero too: 0 * NaN is NaN
    assert torch.isnan(out[bad]).all()
    assert torch.equal(out[~bad], clean[~bad])
    # a weight row of NaN touches its own record slot only
    s2 = scales.clone()
    s2[7] = 255
    y[3], y[150] = 0.0, 1.0
    dcn.predictor_mx(y, codes, s2, None, G=G, K=K, out=out)
    flat = out.view(M, -1)
    slot = int(ow.slots(G, 9)[7])
    assert torch.isnan(flat[:, slot]).all()
    assert torch.isfinite(flat[:, [i for i in range(54) if i != slot]]).all()


def test_predictor_mx_equals_the_projection_of_the_values(cuda_device):
    """The plain predictor on the values read back: same sums up to fp32 rounding."""
    M, C, G, K = 3000, 64, 4, 3
    g = torch.Generator(device=cuda_device).manual_seed(0)
    y = torch.randn(M, C, generator=g, device=cuda_device)
    w = torch.randn(108, C, generator=g, device=cuda_device) / 8
    b = torch.randn(108, generator=g, device=cuda_device)
    wc, ws = dcn.mx_quantize(w)
    yc, ys = dcn.mx_quantize(y)
    a = dcn.predictor_mx(y, wc, ws, b, G=G, K=K)
    yv, wv = dcn.mx_dequantize(yc, ys, C), dcn.mx_dequantize(wc, ws, C)
    r = dcn.predictor(yv, wv, b, G=G, K=K)
    mag = dcn.predictor(yv.abs(), wv.abs(), b.abs(), G=G, K=K)
    assert bool(((a - r).abs() <= 2 * (C + 2) * U * mag).all())


def test_predictor_mx_empty(cuda_device):
    codes, scales, _ = _mx_weight(27, 64, 1, cuda_device)
    y = torch.zeros(0, 7, 64, device=cuda_device, dtype=torch.float16)
    assert dcn.predictor_mx(y, codes, scales, None, G=1, K=3).shape == (0, 7, 1, 27)


# -------------------------------------------------------- predictor backward ---

def _check_grads(grads, y, w, g, G, P, with_bias):
    ref = ow.predictor_backward(_np(y), _np(w), _np(g), G, P)
    mag = ow.predictor_backward(np.abs(_np(y)), np.abs(_np(w)), np.abs(_np(g)), G, P)
    M, NO = y.shape[0], w.shape[0]
    for i, (n, name) in enumerate(((NO, "grad_y"), (M, "grad_weight"), (M, "grad_bias"))):
        if name == "grad_bias" and not with_bias:
            assert grads[2] is None
            continue
        err, tol = np.abs(_np(grads[i]) - ref[i]), (n + 2) * U * mag[i]
        assert np.all(err <= tol), f"{name}: {np.max(err - tol):.3e} over"


BWD_CASES = [
    # M, C, G, K, remove_center, bias
    (1, 64, 4, 3, False, True),
    (129, 64, 4, 3, False, True),
    (1000, 128, 8, 3, False, True),
    (300, 256, 16, 3, False, False),
    (77, 320, 8, 3, True, True),
    (260, 512, 32, 3, False, True),
    (65, 32, 1, 1, False, True),
    (700, 1, 1, 1, False, True),       # one input channel, three outputs
    (200, 33, 3, 3, False, True),
    (131, 100, 5, 3, False, True),
    (513, 9, 2, 5, False, True),
    (4999, 64, 4, 3, False, True),
    (12000, 512, 32, 3, False, True),  # more than one run of tiles per CTA between two readings of the sums
    # at most 64 channels and 128 slots: one or two chunks of slots, channels that end inside a half, several runs
    (1, 8, 4, 1, False, True),
    (300, 24, 4, 3, False, True),
    (257, 56, 8, 2, False, False),
    (20001, 40, 8, 2, False, True),
    (19000, 64, 10, 2, False, True),
    (305000, 16, 5, 2, False, True),
    (304001, 64, 4, 3, False, True),
    (610000, 33, 4, 3, False, True),   # (rows that TMA cannot take)
    (2200, 1024, 44, 3, False, True),  # one CTA per part of the weight, two runs of tiles
    (256, 256, 16, 3, False, True),
]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", BWD_CASES, ids=lambda c: "x".join(map(str, c)))
def test_predictor_backward(case, dtype, cuda_device):
    M, C, G, K, rc, bias = case
    P = K * K - (1 if rc else 0)
    NO = 3 * G * P
    g = torch.Generator().manual_seed(M + C)
    y = (torch.randn(M, C, generator=g) * torch.exp(torch.randn(C, generator=g))).to(TD[dtype])
    w = (torch.randn(NO, C, generator=g) * C ** -0.5).to(TD[dtype])
    gr = torch.randn(M, G, 3 * P, generator=g) * torch.exp(3 * torch.randn(M, 1, 1, generator=g))
    gr[::5] = 0.0
    gy, uy = _guarded((M, C), torch.float32, cuda_device)
    # (a gradient that is not 16-byte aligned takes the way by partial sums)
    gw, uw = _guarded((NO, C), torch.float32, cuda_device, shift=int(M in (129, 257)))
    gb, ub = _guarded((NO,), torch.float32, cuda_device)
    args = (y.to(cuda_device), w.to(cuda_device), gr.to(cuda_device))
    grads = dcn.predictor_backward(*args, G=G, K=K, remove_center=rc, with_bias=bias, grad_y=gy, grad_weight=gw,
                                   grad_bias=gb if bias else None)
    assert dcn.device_status() == 0
    assert uy() and uw() and ub()
    _check_grads(grads, y, w, gr, G, P, bias)
    again = dcn.predictor_backward(*args, G=G, K=K, remove_center=rc, with_bias=bias)
    for a, b in zip(grads, again):
        assert a is None or torch.equal(a, b)   # the sums' order is fixed


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,C,G", [(20000, 128, 8), (30000, 64, 4), (5000, 320, 8)])
def test_predictor_backward_is_the_same_in_every_run(M, C, G, dtype, cuda_device):
    """Many tiles per SM, so that every ring goes round: equal bits, and integers that every sum holds exactly."""
    g = torch.Generator(device=cuda_device).manual_seed(M)
    y = torch.randint(-2, 3, (M, C), generator=g, device=cuda_device).to(TD[dtype])
    w = torch.randint(-2, 3, (27 * G, C), generator=g, device=cuda_device).to(TD[dtype])
    gr = torch.randint(-8, 9, (M, G, 27), generator=g, device=cuda_device).float()
    first = dcn.predictor_backward(y, w, gr, G=G, K=3)
    sl = torch.tensor(ow.slots(G, 9), device=cuda_device)
    gp = gr.double().view(M, -1)[:, sl]
    # |sums| <= M * 16 < 2^24
    assert torch.equal(first[0].double(), gp @ w.double())
    assert torch.equal(first[1].double(), gp.t() @ y.double())
    assert torch.equal(first[2].double(), gp.sum(dim=0))
    for _ in range(10):
        for a, b in zip(dcn.predictor_backward(y, w, gr, G=G, K=3), first):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_predictor_backward_far_apart_magnitudes_and_misaligned_rows(dtype, cuda_device):
    """Gradients from 1e-30 to 1e30 in one call: every sum keeps fp32 precision relative to its own terms."""
    M, C, G, K = 300, 40, 3, 3
    g = torch.Generator().manual_seed(9)
    gr = torch.randn(M, G, 27, generator=g) * 10.0 ** (torch.rand(M, 1, 1, generator=g) * 60 - 30)
    y, _ = _guarded((M, C), TD[dtype], cuda_device, shift=1)
    w, _ = _guarded((81, C), TD[dtype], cuda_device, shift=3)
    grd, _ = _guarded((M, G, 27), torch.float32, cuda_device, shift=1)
    gy, untouched = _guarded((M, C), torch.float32, cuda_device, shift=1)
    y.copy_(torch.randn(M, C, generator=g))
    w.copy_(torch.randn(81, C, generator=g))
    grd.copy_(gr)
    grads = dcn.predictor_backward(y, w, grd, G=G, K=K, grad_y=gy)
    assert untouched()
    _check_grads(grads, y, w, gr, G, 9, True)


def test_predictor_backward_nan_stays_in_its_rows_and_channels(cuda_device):
    M, C, G, K = 260, 64, 2, 3
    g = torch.Generator(device=cuda_device).manual_seed(2)
    y = torch.randn(M, C, generator=g, device=cuda_device).bfloat16()
    w = torch.randn(54, C, generator=g, device=cuda_device).bfloat16()
    gr = torch.randn(M, G, 27, generator=g, device=cuda_device)
    gr[200, 1, 4] = float("nan")
    y[7, 3] = float("nan")
    gy, gw, gb = dcn.predictor_backward(y, w, gr, G=G, K=K)
    rows = torch.isnan(gy).any(dim=1)
    assert rows.nonzero().flatten().tolist() == [200] and torch.isnan(gy[200]).all()
    ch = ow.slots(G, 9).tolist().index(27 + 4)
    assert torch.isnan(gw[:, 3]).all() and torch.isnan(gw[ch]).all()
    keep = torch.ones(54, dtype=torch.bool, device=cuda_device)
    keep[ch] = False
    assert torch.isfinite(gw[keep][:, [c for c in range(C) if c != 3]]).all()
    assert torch.isnan(gb).nonzero().flatten().tolist() == [ch]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("G", [4, 8], ids=["one_chunk", "two_chunks"])
def test_predictor_backward_in_one_pass_nan_and_far_apart_magnitudes(G, dtype, cuda_device):
    """The kernel that reads the records' gradients once (few channels and slots): rows of 1e-30 to 1e30, then
    NaN and infinities, which stay in their rows, channels and slots."""
    M, C, K = 20100, 64, 2
    NO = 3 * G * K * K
    g = torch.Generator().manual_seed(G)
    gr = torch.randn(M, G, 3 * K * K, generator=g) * 10.0 ** (torch.rand(M, 1, 1, generator=g) * 60 - 30)
    y = torch.randn(M, C, generator=g).to(TD[dtype]).to(cuda_device)
    w = torch.randn(NO, C, generator=g).to(TD[dtype]).to(cuda_device)
    gr = gr.to(cuda_device)
    _check_grads(dcn.predictor_backward(y, w, gr, G=G, K=K), y, w, gr, G, K * K, True)
    gr = torch.randn(M, G, 3 * K * K, generator=g).to(cuda_device)
    gr[200, 1, 4] = float("inf")
    y[19999, 3] = float("nan")
    gy, gw, gb = dcn.predictor_backward(y, w, gr, G=G, K=K)
    assert (~torch.isfinite(gy)).any(dim=1).nonzero().flatten().tolist() == [200]
    ch = ow.slots(G, K * K).tolist().index(3 * K * K + 4)
    bad = torch.zeros(NO, C, dtype=torch.bool, device=cuda_device)
    bad[ch] = bad[:, 3] = True
    assert torch.equal(~torch.isfinite(gw), bad)
    assert (~torch.isfinite(gb)).nonzero().flatten().tolist() == [ch]


def test_predictor_backward_without_pixels_writes_zeros(cuda_device):
    y = torch.zeros(0, 64, device=cuda_device)
    gw = torch.full((27, 64), 5.0, device=cuda_device)
    gy, gw2, gb = dcn.predictor_backward(y, torch.ones(27, 64, device=cuda_device),
                                         torch.zeros(0, 1, 27, device=cuda_device), G=1, K=3, grad_weight=gw)
    assert gy.shape == (0, 64) and gw2 is gw
    assert torch.equal(gw, torch.zeros_like(gw)) and torch.equal(gb, torch.zeros_like(gb))


def test_predictor_backward_against_differences(cuda_device):
    """The loss sum(records * g) is linear in y, weight and bias: differences of the fp32 forward give the
    gradients up to the forward's rounding."""
    M, C, G, K = 50, 24, 2, 3
    gen = torch.Generator(device=cuda_device).manual_seed(4)
    y = torch.randn(M, C, generator=gen, device=cuda_device)
    w = torch.randn(54, C, generator=gen, device=cuda_device)
    b = torch.randn(54, generator=gen, device=cuda_device)
    gr = torch.randn(M, G, 27, generator=gen, device=cuda_device)
    grads = dcn.predictor_backward(y, w, gr, G=G, K=K)
    step = 1.0
    for t, grad in zip((y, w, b), grads):
        for i in torch.randint(t.numel(), (6,), generator=torch.Generator().manual_seed(t.numel())).tolist():
            old = t.view(-1)[i].item()
            vals = []
            for d in (step, -step):
                t.view(-1)[i] = old + d
                vals.append(dcn.predictor(y, w, b, G=G, K=K).double() * gr.double())
            t.view(-1)[i] = old
            diff = ((vals[0] - vals[1]).sum() / (2 * step)).item()
            # each record is rounded C + 2 times from terms below 10 in size; 54 * M of them, weighted by |g|
            tol = (C + 2) * U * 10 * C * gr.abs().sum().item() / step
            assert abs(diff - grad.view(-1)[i].item()) <= tol


def test_offsets_past_32_bits(cuda_device):
    """Records of 2^31 - 1 elements at most, more than 2^32 bytes: the last rows equal a call on them alone."""
    if torch.cuda.get_device_properties(cuda_device).total_memory < 60e9:
        pytest.skip("needs 30 GB")
    M, C, G, tail = 9_900_000, 8, 8, 700
    codes, scales, _ = _mx_weight(216, C, 1, cuda_device)
    g = torch.Generator(device=cuda_device).manual_seed(3)
    y = torch.randn(M, C, generator=g, device=cuda_device).half()
    rec = dcn.predictor_mx(y, codes, scales, None, G=G, K=3)
    assert torch.equal(rec[-tail:], dcn.predictor_mx(y[-tail:].contiguous(), codes, scales, None, G=G, K=3))
    del rec
    w = torch.randn(216, C, generator=g, device=cuda_device).half()
    gr = torch.zeros(M, G, 27, device=cuda_device)
    gr[-tail:] = torch.randn(tail, G, 27, generator=g, device=cuda_device)
    gy, gw, gb = dcn.predictor_backward(y, w, gr, G=G, K=3)
    ty, tw, tb = dcn.predictor_backward(y[-tail:].contiguous(), w, gr[-tail:].contiguous(), G=G, K=3)
    assert torch.equal(gy[-tail:], ty) and not gy[:-tail].any()
    for a, b in ((gw, tw), (gb, tb)):   # the pixels are shared out differently: rounding only
        assert bool(((a - b).abs() <= 1e-4 * b.abs().max()).all())


# ------------------------------------------------------ orthogonalised update ---

MUON = (3.4445, -4.7750, 2.0315)
CUBIC = (1.5, -0.5, 0.0)


def _ortho_tolerance(x, steps, co, eps, dtype):
    """(reference, Frobenius tolerance) of each matrix, as derived at the top."""
    a, b, c = co
    ref, tols = [], []
    for X in _np(x).reshape((-1,) + x.shape[-2:]):
        X = X / (np.linalg.norm(X) + eps)
        local, growth, r = [2 * U * np.linalg.norm(X)], [], 1.0
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
        ref.append(X)
        tols.append(total + HALF_UNIT[dtype] * np.linalg.norm(X) + TINY[dtype] * np.sqrt(X.size))
    return np.stack(ref), tols


def _check_ortho(got, x, steps, co, eps, dtype):
    ref, tols = _ortho_tolerance(x, steps, co, eps, dtype)
    assert got.dtype == x.dtype and got.shape == x.shape
    g = _np(got).reshape(ref.shape)
    for i in range(len(ref)):
        err = np.linalg.norm(g[i] - ref[i])
        assert err <= tols[i], f"matrix {i}: {err:.3e} > {tols[i]:.3e} (norm {np.linalg.norm(ref[i]):.3e})"


ORTHO_CASES = [
    # B, R, C
    (1, 1, 1), (3, 1, 7), (3, 9, 1), (2, 5, 8), (4, 108, 64), (2, 64, 64), (3, 65, 63), (2, 33, 130), (1, 216, 128),
    (3, 256, 432), (1, 192, 320), (2, 129, 257), (1, 864, 512), (5, 40, 600), (70, 12, 10), (1, 640, 640),
]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("co", [MUON, CUBIC], ids=["muon", "cubic"])
@pytest.mark.parametrize("shape", ORTHO_CASES, ids=lambda c: "x".join(map(str, c)))
def test_orthogonalize(shape, co, dtype, cuda_device):
    g = torch.Generator().manual_seed(sum(shape))
    x = (torch.randn(*shape, generator=g) * 0.01).to(TD[dtype])
    out, untouched = _guarded(shape, TD[dtype], cuda_device)
    xd = x.to(cuda_device)
    assert dcn.orthogonalize(xd, coefficients=co, out=out) is out
    assert dcn.device_status() == 0
    assert untouched() and torch.equal(xd.cpu(), x)
    _check_ortho(out, x, 5, co, 1e-7, dtype)
    assert torch.equal(dcn.orthogonalize(xd, coefficients=co), out)


@pytest.mark.parametrize("shape", [(2, 5, 8), (3, 108, 64), (2, 129, 257), (1, 300, 128), (1, 60, 384), (1, 64, 385)],
                         ids=lambda c: "x".join(map(str, c)))
def test_orthogonalize_one_kernel_per_product(shape, cuda_device, monkeypatch):
    """Matrices that one CTA holds, through the kernels of the larger ones too."""
    x = torch.randn(*shape, generator=torch.Generator().manual_seed(5))
    for form in ("", "products"):
        monkeypatch.setenv("DCNV4_ORTHO_FORM", form)
        out = dcn.orthogonalize(x.to(cuda_device))
        assert dcn.device_status() == 0
        _check_ortho(out, x, 5, MUON, 1e-7, "f32")


@pytest.mark.parametrize("steps", [0, 1, 2, 12])
def test_orthogonalize_steps_leading_shape_and_misaligned_rows(steps, cuda_device):
    g = torch.Generator().manual_seed(steps)
    x, _ = _guarded((2, 3, 20, 31), torch.float32, cuda_device, shift=1)
    x.copy_(torch.randn(2, 3, 20, 31, generator=g))
    out, untouched = _guarded((2, 3, 20, 31), torch.float32, cuda_device, shift=3)
    dcn.orthogonalize(x, steps=steps, coefficients=(1.875, -1.25, 0.375), out=out)
    assert untouched()
    _check_ortho(out, x, steps, (1.875, -1.25, 0.375), 1e-7, "f32")
    one = dcn.orthogonalize(x[0, 0].contiguous(), steps=steps, coefficients=(1.875, -1.25, 0.375))
    assert one.shape == (20, 31) and torch.equal(one, out[0, 0])   # a matrix does not depend on its stack


@pytest.mark.parametrize("shape", [(6, 16, 24), (6, 150, 140)], ids=["small", "tiles"])
def test_orthogonalize_zero_nan_and_extreme_matrices(shape, cuda_device):
    """Zero and non-finite matrices keep to themselves; the norm neither overflows nor vanishes."""
    g = torch.Generator().manual_seed(0)
    x = torch.randn(*shape, generator=g)
    x[1] = 0.0
    x[2, 3, 5] = float("nan")
    x[3, 0, 0] = float("inf")
    x[4] *= 1e30
    x[5] *= 1e-30
    out = dcn.orthogonalize(x.to(cuda_device), eps=1e-38)
    assert torch.equal(out[1].cpu(), torch.zeros(shape[1:]))
    assert torch.isnan(out[2]).all() and torch.isnan(out[3]).all()
    keep = [0, 4, 5]
    _check_ortho(out[keep], x[keep], 5, MUON, 1e-38, "f32")
    # a norm far below eps: the division by eps leaves a small matrix
    tiny = torch.randn(1, *shape[1:], generator=g) * 1e-9
    _check_ortho(dcn.orthogonalize(tiny.to(cuda_device), eps=1.0), tiny, 5, MUON, 1.0, "f32")


def test_orthogonalize_low_rank(cuda_device):
    """Rank 3 of 64: the other singular values stay at rounding size."""
    g = torch.Generator().manual_seed(6)
    x = torch.matmul(torch.randn(2, 64, 3, generator=g), torch.randn(2, 3, 96, generator=g))
    out = dcn.orthogonalize(x.to(cuda_device))
    _check_ortho(out, x, 5, MUON, 1e-7, "f32")
    s = np.linalg.svd(_np(out), compute_uv=False)
    assert np.all((s[:, :3] > 0.6) & (s[:, :3] < 1.25))


@pytest.mark.parametrize("shape", [(2, 78, 10), (10, 318, 124), (1, 809, 840)], ids=lambda c: "x".join(map(str, c)))
def test_orthogonalize_keeps_the_accuracy_of_fp32_products(shape, cuda_device):
    """The relative error (Frobenius) is at most half as large again as that of the same iteration by fp32 matrix
    products: an operand of 22 bits is off by up to 2 units of fp32's 24 in the worst octave, 1.5 in the mean square."""
    g = torch.Generator(device=cuda_device).manual_seed(31)
    x = torch.randn(shape, generator=g, device=cuda_device)

    def plain(t):
        v = t.transpose(-1, -2) if shape[1] > shape[2] else t
        v = v / (torch.linalg.matrix_norm(v, keepdim=True) + 1e-7)
        for _ in range(5):
            a = v @ v.transpose(-1, -2)
            v = MUON[0] * v + (MUON[1] * a + MUON[2] * (a @ a)) @ v
        return v.transpose(-1, -2) if shape[1] > shape[2] else v
    ref = plain(x.double())
    err = [float((t.double() - ref).norm() / ref.norm()) for t in (dcn.orthogonalize(x), plain(x))]
    assert err[0] <= 1.5 * err[1] + 1e-7, err


def test_orthogonalize_refuses_unbounded_coefficients(cuda_device):
    x = torch.randn(4, 4, device=cuda_device)
    with pytest.raises(dcn.DCNv4Error, match="COEFFICIENTS"):
        dcn.orthogonalize(x, coefficients=(5.0, 0.0, 0.0))
    with pytest.raises(ValueError):
        dcn.orthogonalize(x, out=torch.empty(4, 5, device=cuda_device))
    assert dcn.orthogonalize(x[None][:0]).shape == (0, 4, 4)


# ------------------------------------------------------------ used together ---

def _calls(dev):
    g = torch.Generator(device=dev).manual_seed(11)
    y = torch.randn(700, 64, generator=g, device=dev).half()
    w = (torch.randn(108, 64, generator=g, device=dev) / 8).half()
    gr = torch.randn(700, 4, 27, generator=g, device=dev)
    b = torch.randn(108, generator=g, device=dev)
    m = torch.randn(3, 108, 64, generator=g, device=dev)
    big = torch.randn(2, 300, 200, generator=g, device=dev)

    def run():
        codes, scales = dcn.mx_quantize(w)
        return (dcn.mx_dequantize(codes, scales, 64), dcn.predictor_mx(y, codes, scales, b, G=4, K=3),
                *dcn.predictor_backward(y, w, gr, G=4, K=3), dcn.orthogonalize(m), dcn.orthogonalize(big))
    return run, (y, w, gr, b, m, big)


def test_on_another_stream_and_two_at_once(cuda_device):
    run, _ = _calls(cuda_device)
    want = run()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(run())
    torch.cuda.synchronize()
    for r in got:
        for a, b in zip(r, want):
            assert torch.equal(a, b)


def test_tensor_memory_shared_between_streams(cuda_device):
    """Projections that want all of an SM's tensor memory, each followed by one that wants little, beside a second
    stream whose small kernels hold columns nearly all the time: everything finishes, with the same results."""
    g = torch.Generator(device=cuda_device).manual_seed(4)
    y = torch.randn(60000, 64, generator=g, device=cuda_device).half()
    w = (torch.randn(216, 64, generator=g, device=cuda_device) / 8).half()
    codes, scales = dcn.mx_quantize(w)
    small = dcn.mx_quantize((torch.randn(27, 64, generator=g, device=cuda_device) / 8).half())
    torch.cuda.synchronize()

    def main():
        return dcn.predictor(y, w, None, G=8, K=3), dcn.predictor_mx(y[:9000], codes, scales, None, G=8, K=3)

    def side():
        return (dcn.predictor_mx(y, *small, None, G=1, K=3),)
    want_main, want_side = main(), side()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(10):
        for s, call, want in zip(streams, (main, side), (want_main, want_side)):
            with torch.cuda.stream(s):
                got.append((call(), want))
    torch.cuda.synchronize()
    for r, want in got:
        for a, b in zip(r, want):
            assert torch.equal(a, b)
    assert binding.device_status() == 0


@pytest.mark.parametrize("M", [130, 20000])
def test_gradients_are_complete_for_the_next_launch(M, cuda_device):
    """The next kernel on the stream reads every gradient at once, eagerly and in a graph: kernels that start
    before the one in front of them has finished must still leave everything complete."""
    g = torch.Generator(device=cuda_device).manual_seed(M)
    y = torch.randn(M, 128, generator=g, device=cuda_device).bfloat16()
    w = torch.randn(216, 128, generator=g, device=cuda_device).bfloat16()
    gr = torch.randn(M, 8, 27, generator=g, device=cuda_device)
    outs = [torch.empty(M, 128, device=cuda_device), torch.empty(216, 128, device=cuda_device),
            torch.empty(216, device=cuda_device)]

    def run():
        for t in outs:
            t.fill_(float("nan"))
        dcn.predictor_backward(y, w, gr, G=8, K=3, grad_y=outs[0], grad_weight=outs[1], grad_bias=outs[2])
        return [dcn.mx_quantize(t) for t in outs]

    first = run()
    torch.cuda.synchronize()
    want = [dcn.mx_quantize(t) for t in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run()
    for _ in range(20):
        for got in (run(), captured):
            graph.replay()
            for a, b in zip(got, want):
                assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    for a, b in zip(first, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_stream_argument(cuda_device):
    x = torch.randn(2, 80, 50, device=cuda_device)
    want = dcn.orthogonalize(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = dcn.orthogonalize(x, stream=s)
    codes, scales = dcn.mx_quantize(x, stream=s)
    back = dcn.mx_dequantize(codes, scales, 50, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    c2, s2 = dcn.mx_quantize(x)
    assert torch.equal(codes, c2) and torch.equal(scales, s2) and torch.equal(back, dcn.mx_dequantize(c2, s2, 50))


def test_captured_and_replayed(cuda_device):
    """Two graphs of the same calls, replayed in turn on new inputs."""
    run, inputs = _calls(cuda_device)
    run()   # kernel attributes are set outside the capture
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        gph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gph):
            outs = run()
        graphs.append((gph, outs))
    for seed in range(3):
        gen = torch.Generator(device=cuda_device).manual_seed(seed)
        for t in inputs:
            t.copy_(torch.randn(t.shape, generator=gen, device=cuda_device))
        for gph, _ in graphs:
            gph.replay()
        want = run()
        torch.cuda.synchronize()
        for _, outs in graphs:
            for a, b in zip(outs, want):
                assert torch.equal(a, b)


def test_a_training_step_of_the_predictor_and_its_four_bit_form(cuda_device):
    """predictor -> forward -> backward -> predictor_backward -> orthogonalised update of the weight ->
    the updated weight quantised once -> predictor_mx -> forward; each stage against its fp64 definition on the
    stage's own inputs."""
    N, H, C, G, K = 2, 16, 64, 4, 3
    P, lr = K * K, 0.02
    gen = torch.Generator(device=cuda_device).manual_seed(21)
    x = torch.randn(N, H, H, C, generator=gen, device=cuda_device).half()
    y = torch.randn(N, H, H, C, generator=gen, device=cuda_device).half()
    master = torch.randn(3 * G * P, C, generator=gen, device=cuda_device) * 0.1
    bias = torch.randn(3 * G * P, generator=gen, device=cuda_device) * 0.5
    go = torch.randn(N, H, H, C, generator=gen, device=cuda_device).half()
    w = master.half()
    rec = dcn.predictor(y, w, bias, G=G, K=K)
    dcn.forward(x, rec, G=G, K=K, pad=1)
    _, grec = dcn.backward(x, rec, go, G=G, K=K, pad=1)
    gy, gw, gb = dcn.predictor_backward(y, w, grec, G=G, K=K)
    assert gy.shape == y.shape
    _check_grads((gy.view(-1, C), gw, gb), y.view(-1, C), w, grec.view(-1, G, 3 * P), G, P, True)
    update = dcn.orthogonalize(gw)
    _check_ortho(update, gw, 5, MUON, 1e-7, "f32")
    new = master - lr * update
    codes, scales = dcn.mx_quantize(new)
    rc, rs = ow.mx_quantize(_np(new))
    assert np.array_equal(ow.mx_unpack(codes.cpu().numpy()), rc) and np.array_equal(scales.cpu().numpy(), rs)
    rec4 = dcn.predictor_mx(y, codes, scales, bias, G=G, K=K)
    _check_mx_projection(rec4, y.view(-1, C), ow.mx_values(rc, rs, C), bias.double().cpu().numpy(), G, P, "f16")
    out = dcn.forward(x, rec4, G=G, K=K, pad=1)
    ref = oracle.dcnv4_forward(_np(x), _np(rec4), G=G, K=K, pad=1)
    assert np.abs(_np(out) - ref).max() <= 4e-3 * np.abs(ref).max()
    assert binding.device_status() == 0
