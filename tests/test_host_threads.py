"""Calls from host threads that have not used CUDA before."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


def _in_new_thread(f):
    got = []

    def work():
        try:
            got.append(f())
        except Exception as e:  # handed to the caller below
            got.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    if isinstance(got[0], Exception):
        raise got[0]
    return got[0]


def test_product_from_a_new_thread(cuda_lib):
    """The tensor maps need a current context, which a new thread has not."""
    a, = cuda_lib.kda_fp8_quantize(torch.randn(70, 256, device="cuda"))
    b, = cuda_lib.kda_fp8_quantize(torch.randn(200, 256, device="cuda"), "tile")
    want = cuda_lib.kda_fp8_matmul(a, b)
    out = torch.empty_like(want)
    _in_new_thread(lambda: cuda_lib.kda_fp8_matmul(a, b, out=out))
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    got = _in_new_thread(lambda: cuda_lib.kda_fp8_matmul(a, b))
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_forward_and_backward_from_new_threads(cuda_lib):
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v, d = (torch.randn(1, 128, 2, 128, device="cuda", generator=g).bfloat16() for _ in range(4))
    gate = -torch.rand(1, 128, 2, 128, device="cuda", generator=g)
    beta = torch.rand(1, 128, 2, device="cuda", generator=g)
    want = cuda_lib.kda_chunk_fwd(q, k, v, gate, beta)
    grads = cuda_lib.kda_chunk_bwd(q, k, v, gate, beta, d)
    got = _in_new_thread(lambda: cuda_lib.kda_chunk_fwd(q, k, v, gate, beta))
    got_grads = _in_new_thread(lambda: cuda_lib.kda_chunk_bwd(q, k, v, gate, beta, d))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert all(torch.equal(got_grads[n], t) for n, t in grads.items() if t is not None)
