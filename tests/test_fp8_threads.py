"""The 8-bit projection path called by several host threads at once."""
import ctypes
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


def _run(bodies):
    """Each body in a thread of its own, started together; raises what one raised."""
    errors, start = [], threading.Barrier(len(bodies))

    def work(body):
        try:
            start.wait()
            body()
        except BaseException as e:  # noqa: B902
            errors.append(e)

    threads = [threading.Thread(target=work, args=(b,)) for b in bodies]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if errors:
        raise errors[0]


def test_sizes_that_need_different_shared_memory(cuda_lib):
    """The same kernels at sizes that need different amounts of shared memory,
    called from eight threads at once, each on a stream of its own: no call is
    refused, and the results are those of a call alone."""
    lib, k = cuda_lib.load_library(), cuda_lib
    counts, bodies, checks, keep = [], [], [], []

    def add(f, args, out, want):
        stream = torch.cuda.Stream()
        counts.append(0)
        i, p = len(counts) - 1, ctypes.byref(args)

        def body():
            for _ in range(3000):
                counts[i] += f(p, stream.cuda_stream) != k.KDA_OK

        keep.append((args, stream))
        bodies.append(body)
        checks.append((out, want))

    for cols in (4096, 8192) * 2:  # 64 and 128 KB
        x = torch.randn(1, cols, device="cuda")
        h, out = torch.empty_like(x), torch.empty_like(x)
        add(lib.kda_rms_norm, k.kda_rms_norm_args(1, cols, k.KDA_F32, x.data_ptr(), x.data_ptr(), None, 1e-6, h.data_ptr(),
                                                  out.data_ptr()), out, k.kda_rms_norm(x, None, x).out)
        keep.append((x, h))
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    for m, n, kk in ((1, 256, 256), (64, 256, 8192)) * 2:  # the least, and all of an SM
        a, = k.kda_fp8_quantize(torch.randn(m, kk, device="cuda"))
        b, = k.kda_fp8_quantize(torch.randn(n, kk, device="cuda"), "tile")
        want = k.kda_fp8_matmul(a, b)
        out = torch.empty_like(want)
        add(lib.kda_fp8_matmul, k.kda_fp8_matmul_args(m, n, kk, k.KDA_FP8_NT, a.data.data_ptr(), kk, a.scales.data_ptr(),
                                                      b.data.data_ptr(), kk, b.scales.data_ptr(), out.data_ptr(), n,
                                                      k.KDA_BF16, ws.data_ptr(), 256, 0), out, want)
        keep.append((a, b))
    torch.cuda.synchronize()
    _run(bodies)
    torch.cuda.synchronize()
    assert counts == [0] * len(counts), "refused calls"
    assert all(torch.equal(o, w) for o, w in checks)
