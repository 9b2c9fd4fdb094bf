"""The first call that a process ever makes of each operator around the predictor's weight may be a captured one."""
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

PROGRAM = """
import torch
import deformable_convolution_sparse_b200 as dcn
g = torch.Generator(device="cuda").manual_seed(1)
rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
y, w, gr, m, big = rand(700, 64).half(), (rand(108, 64) / 8).half(), rand(700, 4, 27), rand(3, 108, 64), rand(2, 300, 200)


def run():
    codes, scales = dcn.mx_quantize(w)
    return [codes, scales, dcn.mx_dequantize(codes, scales, 64), dcn.predictor_mx(y, codes, scales, None, G=4, K=3),
            *dcn.predictor_backward(y, w, gr, G=4, K=3), *dcn.predictor_backward(y.float(), w.float(), gr, G=4, K=3),
            dcn.orthogonalize(m), dcn.orthogonalize(big)]


y.float(), w.float()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    outs = run()
graph.replay()
torch.cuda.synchronize()
for a, b in zip(outs, run()):
    assert torch.equal(a, b)
assert dcn.device_status() == 0
print("first calls captured")
"""


def test_first_calls_captured(cuda_device):
    r = subprocess.run([sys.executable, "-c", PROGRAM], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "first calls captured" in r.stdout, r.stderr[-2000:]
