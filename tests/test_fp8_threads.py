"""The 8-bit projection path called by several host threads at once, and
for the first time during a stream capture."""
import ctypes
import os
import subprocess
import sys
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


def test_threads_share_one_error_word(cuda_lib):
    """Threads that make a device's first products together use the same
    error word: a report in it is not lost, and none of them holds memory that
    was let go of."""
    dev = torch.cuda.current_device()
    for _ in range(20):
        cuda_lib._fp8_status_words.clear()
        got = []
        _run([lambda: got.append(cuda_lib._fp8_status_word(dev))] * 6)
        assert len(set(got)) == 1
    assert cuda_lib.kda_fp8_matmul_status() == cuda_lib.KDA_OK


_FIRST_CALLS_IN_A_CAPTURE = """
import sys
import torch
sys.path.insert(0, sys.argv[1])
import chunked_kimi_delta_gb300 as kda
x = torch.randn(300, 1024, device="cuda").bfloat16()
w = torch.randn(1024, 1024, device="cuda")

def layer():
    n = kda.kda_rms_norm(x, None, x, fp8=True)
    w8, = kda.kda_fp8_quantize(w, "tile")
    y = kda.kda_fp8_matmul(n.fp8, w8)
    d_row, d_col = kda.kda_fp8_quantize(y, ("row", "col"))
    n_col, = kda.kda_fp8_quantize(n.out, "col")
    dw = kda.kda_fp8_matmul(d_col, n_col, "tn", out_dtype=torch.float32)
    dx, dweight = kda.kda_rms_norm_bwd(kda.kda_fp8_matmul(d_row, w8, "nn"), n.residual_out)
    return n.out, n.residual_out, y, dw, dx, dweight

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = layer()
for seed in (1, 2):
    x.copy_(torch.randn(x.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, layer()))
assert kda.kda_fp8_matmul_status() == kda.KDA_OK
print("same")
"""


def test_first_calls_of_a_process_in_a_capture(cuda_lib):
    """Norm, quantiser and products whose first call is recorded into a graph:
    replayed on other inputs they give what calls outside give, bit for bit."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(cuda_lib.__file__)))
    r = subprocess.run([sys.executable, "-c", _FIRST_CALLS_IN_A_CAPTURE, root], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr
