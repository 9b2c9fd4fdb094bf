"""The operators around the predictor's weight from several host threads at once, a stream each."""
import threading

import pytest
import torch

import deformable_convolution_sparse_b200 as dcn

pytestmark = pytest.mark.gpu


def test_four_threads_a_stream_each(cuda_device):
    g = torch.Generator(device=cuda_device).manual_seed(3)
    y = torch.randn(3000, 64, generator=g, device=cuda_device).half()
    w = (torch.randn(108, 64, generator=g, device=cuda_device) / 8).half()
    gr = torch.randn(3000, 4, 27, generator=g, device=cuda_device)
    m = torch.randn(3, 108, 64, generator=g, device=cuda_device)
    big = torch.randn(2, 300, 200, generator=g, device=cuda_device)
    y32, w32 = y.float(), w.float()

    def run():
        codes, scales = dcn.mx_quantize(w)
        return [codes, scales, dcn.mx_dequantize(codes, scales, 64), dcn.predictor_mx(y, codes, scales, None, G=4, K=3),
                *dcn.predictor_backward(y, w, gr, G=4, K=3), *dcn.predictor_backward(y32, w32, gr, G=4, K=3),
                dcn.orthogonalize(m), dcn.orthogonalize(big)]

    want = run()
    torch.cuda.synchronize()
    wrong = []

    def work(n):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(20):
                    got = run()
                    s.synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want)):
                        wrong.append(n)
        except Exception as e:  # noqa: BLE001 (shown by the assertion)
            wrong.append(repr(e))

    threads = [threading.Thread(target=work, args=(n,)) for n in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong[:3]
    assert dcn.device_status() == 0
