"""Host-side tests (no GPU) of the operators around the predictor's weight: every
error class is reported before any CUDA call, empty calls touch nothing, and the
workspaces' sizes depend on the arguments alone."""
import ctypes
import glob
import os
import re

import pytest

from deformable_convolution_sparse_b200 import binding as B

# fake, never dereferenced device addresses
X, CODES, SCALES, OUT, BIAS, WS = (0x10000000 * k for k in (1, 2, 3, 4, 5, 6))
GY, GW, GB = 0x70000000, 0x80000000, 0x90000000
NAN, INF = float("nan"), float("inf")


def _q(x=X, c=CODES, s=SCALES, M=100, C=64, dtype=B.DCNV4_F16):
    return B.load_library().dcnv4_mx_quantize(x, c, s, M, C, dtype, None)


def _dq(x=X, c=CODES, s=SCALES, M=100, C=64, dtype=B.DCNV4_F16):
    return B.load_library().dcnv4_mx_dequantize(c, s, x, M, C, dtype, None)


@pytest.mark.parametrize("call", [_q, _dq], ids=["quantize", "dequantize"])
@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), "DCNV4_ERR_SHAPE"), (dict(C=0), "DCNV4_ERR_SHAPE"), (dict(dtype=3), "DCNV4_ERR_DTYPE"),
    (dict(x=0), "DCNV4_ERR_NULL"), (dict(c=0), "DCNV4_ERR_NULL"), (dict(s=0), "DCNV4_ERR_NULL"),
    (dict(x=X + 1), "DCNV4_ERR_ALIGN"), (dict(c=CODES + 8), "DCNV4_ERR_ALIGN"),
    (dict(x=X + 2, dtype=B.DCNV4_F32), "DCNV4_ERR_ALIGN"),
    (dict(c=X + 64), "DCNV4_ERR_ALIAS"), (dict(s=X + 1), "DCNV4_ERR_ALIAS"),
    (dict(M=1 << 26, C=1), "DCNV4_ERR_TOO_LARGE"),   # one channel takes a whole block of 32
    (dict(M=1, C=(1 << 31) - 1), "DCNV4_ERR_TOO_LARGE"),
])
def test_mx_reports_each_error_class(call, kw, status):
    assert call(**kw) == B.STATUS[status]


def test_mx_quantize_outputs_must_not_overlap_and_empty_calls_touch_nothing():
    assert _q(s=CODES + 5) == B.STATUS["DCNV4_ERR_ALIAS"]
    assert _q(x=0, c=0, s=0, M=0) == B.DCNV4_OK
    assert _dq(x=0, c=0, s=0, M=0) == B.DCNV4_OK


def _pmx(y=X, c=CODES, s=SCALES, b=BIAS, rec=OUT, M=1000, C=64, G=4, K=3, flags=0, dtype=B.DCNV4_F16):
    return B.load_library().dcnv4_predictor_mx(y, c, s, b, rec, M, C, G, K, flags, dtype, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), "DCNV4_ERR_SHAPE"), (dict(C=0), "DCNV4_ERR_SHAPE"), (dict(G=0), "DCNV4_ERR_SHAPE"),
    (dict(K=17), "DCNV4_ERR_SHAPE"), (dict(K=2, flags=B.FLAG_REMOVE_CENTER), "DCNV4_ERR_SHAPE"),
    (dict(flags=B.FLAG_SOFTMAX), "DCNV4_ERR_FLAGS"), (dict(dtype=9), "DCNV4_ERR_DTYPE"),
    (dict(y=0), "DCNV4_ERR_NULL"), (dict(c=0), "DCNV4_ERR_NULL"), (dict(s=0), "DCNV4_ERR_NULL"),
    (dict(rec=0), "DCNV4_ERR_NULL"),
    (dict(y=X + 1), "DCNV4_ERR_ALIGN"), (dict(c=CODES + 4), "DCNV4_ERR_ALIGN"), (dict(b=BIAS + 2), "DCNV4_ERR_ALIGN"),
    (dict(rec=OUT + 1), "DCNV4_ERR_ALIGN"),
    (dict(rec=X + 64), "DCNV4_ERR_ALIAS"), (dict(rec=CODES), "DCNV4_ERR_ALIAS"), (dict(rec=SCALES), "DCNV4_ERR_ALIAS"),
    (dict(b=OUT + 16), "DCNV4_ERR_ALIAS"),
    (dict(M=1 << 25, C=128), "DCNV4_ERR_TOO_LARGE"), (dict(M=1 << 26, C=1, G=1, K=1), "DCNV4_ERR_TOO_LARGE"),
])
def test_predictor_mx_reports_each_error_class(kw, status):
    assert _pmx(**kw) == B.STATUS[status]


def test_predictor_mx_empty_batch_touches_nothing():
    assert _pmx(y=0, c=0, s=0, b=0, rec=0, M=0) == B.DCNV4_OK


def _bws(M=1000, C=64, G=4, K=3, flags=0, dtype=B.DCNV4_F16):
    v = ctypes.c_size_t(0)
    rc = B.load_library().dcnv4_predictor_backward_workspace(M, C, G, K, flags, dtype, ctypes.byref(v))
    return rc, v.value


def _pb(y=X, w=CODES, g=SCALES, gy=GY, gw=GW, gb=GB, ws=WS, size=None, M=1000, C=64, G=4, K=3, flags=0,
        dtype=B.DCNV4_F16):
    if size is None:
        size = _bws(M, C, G, K, flags, dtype)[1]
    return B.load_library().dcnv4_predictor_backward(y, w, g, gy, gw, gb, ws, size, M, C, G, K, flags, dtype, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), "DCNV4_ERR_SHAPE"), (dict(C=0), "DCNV4_ERR_SHAPE"), (dict(G=0), "DCNV4_ERR_SHAPE"),
    (dict(K=0), "DCNV4_ERR_SHAPE"), (dict(K=4, flags=B.FLAG_REMOVE_CENTER), "DCNV4_ERR_SHAPE"),
    (dict(flags=B.FLAG_CENTER_SCALE), "DCNV4_ERR_FLAGS"), (dict(dtype=-1), "DCNV4_ERR_DTYPE"),
    (dict(y=0), "DCNV4_ERR_NULL"), (dict(w=0), "DCNV4_ERR_NULL"), (dict(g=0), "DCNV4_ERR_NULL"),
    (dict(gy=0), "DCNV4_ERR_NULL"), (dict(gw=0), "DCNV4_ERR_NULL"), (dict(ws=0), "DCNV4_ERR_NULL"),
    (dict(y=X + 1), "DCNV4_ERR_ALIGN"), (dict(g=SCALES + 2), "DCNV4_ERR_ALIGN"), (dict(gw=GW + 2), "DCNV4_ERR_ALIGN"),
    (dict(gb=GB + 1), "DCNV4_ERR_ALIGN"), (dict(ws=WS + 8), "DCNV4_ERR_ALIGN"),
    (dict(size=0), "DCNV4_ERR_WORKSPACE"), (dict(size=1000), "DCNV4_ERR_WORKSPACE"),
    (dict(gy=X), "DCNV4_ERR_ALIAS"), (dict(gw=CODES), "DCNV4_ERR_ALIAS"), (dict(gb=SCALES + 64), "DCNV4_ERR_ALIAS"),
    (dict(gw=GY + 64), "DCNV4_ERR_ALIAS"), (dict(gb=GW), "DCNV4_ERR_ALIAS"), (dict(ws=GY), "DCNV4_ERR_ALIAS"),
    (dict(ws=X), "DCNV4_ERR_ALIAS"),
    (dict(M=1 << 25, C=128), "DCNV4_ERR_TOO_LARGE"),
])
def test_predictor_backward_reports_each_error_class(kw, status):
    assert _pb(**kw) == B.STATUS[status]


def test_predictor_backward_workspace():
    assert _bws(M=0) == (B.DCNV4_OK, 0)
    rc, one = _bws(M=1)
    assert rc == B.DCNV4_OK and one > 0
    assert _bws(C=0)[0] == B.STATUS["DCNV4_ERR_SHAPE"]
    assert B.load_library().dcnv4_predictor_backward_workspace(1, 64, 4, 3, 0, 1, None) == B.STATUS["DCNV4_ERR_NULL"]


def _ows(Bn=2, R=108, C=64, dtype=B.DCNV4_F32):
    v = ctypes.c_size_t(0)
    rc = B.load_library().dcnv4_orthogonalize_workspace(Bn, R, C, dtype, ctypes.byref(v))
    return rc, v.value


def _o(x=X, out=OUT, ws=WS, size=None, Bn=2, R=108, C=64, steps=5, a=3.4445, b=-4.775, c=2.0315, eps=1e-7,
       dtype=B.DCNV4_F32):
    if size is None:
        size = _ows(Bn, R, C, dtype)[1]
    return B.load_library().dcnv4_orthogonalize(x, out, ws, size, Bn, R, C, steps, a, b, c, eps, dtype, None)


@pytest.mark.parametrize("kw,status", [
    (dict(Bn=-1), "DCNV4_ERR_SHAPE"), (dict(R=0), "DCNV4_ERR_SHAPE"), (dict(C=-3), "DCNV4_ERR_SHAPE"),
    (dict(steps=-1), "DCNV4_ERR_SHAPE"), (dict(steps=65), "DCNV4_ERR_SHAPE"), (dict(dtype=3), "DCNV4_ERR_DTYPE"),
    (dict(a=NAN), "DCNV4_ERR_COEFFICIENTS"), (dict(b=INF), "DCNV4_ERR_COEFFICIENTS"),
    (dict(eps=0.0), "DCNV4_ERR_COEFFICIENTS"), (dict(eps=-1.0), "DCNV4_ERR_COEFFICIENTS"),
    (dict(eps=NAN), "DCNV4_ERR_COEFFICIENTS"),
    (dict(a=5.0, b=0.0, c=0.0, steps=1), "DCNV4_ERR_COEFFICIENTS"),     # a singular value of 1 becomes 5
    (dict(a=1.1, b=0.0, c=0.0, steps=20), "DCNV4_ERR_COEFFICIENTS"),    # 1.1^20 is above 4
    (dict(a=100.0, b=-100.0, c=0.0, steps=1), "DCNV4_ERR_COEFFICIENTS"),
    (dict(x=0), "DCNV4_ERR_NULL"), (dict(out=0), "DCNV4_ERR_NULL"), (dict(ws=0), "DCNV4_ERR_NULL"),
    (dict(x=X + 2), "DCNV4_ERR_ALIGN"), (dict(out=OUT + 1), "DCNV4_ERR_ALIGN"), (dict(ws=WS + 16), "DCNV4_ERR_ALIGN"),
    (dict(size=100), "DCNV4_ERR_WORKSPACE"),
    (dict(out=X), "DCNV4_ERR_ALIAS"), (dict(ws=X), "DCNV4_ERR_ALIAS"), (dict(out=WS + 256), "DCNV4_ERR_ALIAS"),
    (dict(R=1 << 16, C=1 << 16, Bn=1), "DCNV4_ERR_TOO_LARGE"), (dict(Bn=1 << 20, R=64, C=64), "DCNV4_ERR_TOO_LARGE"),
])
def test_orthogonalize_reports_each_error_class(kw, status):
    if kw.get("Bn", 1) < 0 or kw.get("R", 1) <= 0 or kw.get("C", 1) <= 0 or status == "DCNV4_ERR_TOO_LARGE" or \
            kw.get("dtype", 0) == 3:
        kw = dict(kw, size=1 << 40)
    assert _o(**kw) == B.STATUS[status]


def test_orthogonalize_empty_stack_and_workspace():
    assert _o(x=0, out=0, ws=0, Bn=0) == B.DCNV4_OK
    assert _ows(Bn=0) == (B.DCNV4_OK, 0)
    assert _ows()[1] > 0
    assert B.load_library().dcnv4_orthogonalize_workspace(2, 8, 8, 0, None) == B.STATUS["DCNV4_ERR_NULL"]


def test_bindings_refuse_cpu_tensors_and_wrong_arguments():
    import torch
    x = torch.zeros(4, 64)
    c, s = torch.zeros(27, 32, dtype=torch.uint8), torch.zeros(27, 2, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        B.mx_quantize(x)
    with pytest.raises(ValueError, match="CUDA"):
        B.mx_dequantize(c, s, 64)
    with pytest.raises(TypeError):
        B.mx_dequantize(c, s, 64, torch.float64)
    with pytest.raises(ValueError, match="CUDA"):
        B.predictor_mx(x, c, s, None, G=1, K=3)
    with pytest.raises(ValueError, match="CUDA"):
        B.predictor_backward(x, torch.zeros(27, 64), torch.zeros(4, 1, 27), G=1, K=3)
    with pytest.raises(ValueError, match="CUDA"):
        B.orthogonalize(x)


def test_tensor_memory_is_held_before_the_next_launch_may_start():
    """Every kernel that allocates tensor memory passes a CTA barrier between that and letting the next launch
    start; else a CTA still waiting for columns (another stream's kernel has them) could see the next launch's CTA
    take them and wait for this kernel in turn, for good."""
    csrc = os.path.join(os.path.dirname(B.__file__), "csrc")
    seen = 0
    for path in sorted(glob.glob(os.path.join(csrc, "*.cuh"))):
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for kernel in text.split("__global__")[1:]:
            alloc = re.search(r"tc::alloc\(|tcgen05\.alloc", kernel)
            trigger = kernel.find("griddepcontrol.launch_dependents")
            if alloc and trigger >= 0:
                seen += 1
                assert "__syncthreads();" in kernel[alloc.start():trigger], (os.path.basename(path), kernel[:120])
    assert seen >= 6
