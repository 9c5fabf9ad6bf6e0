"""The 8-bit projection path at the ends of fp32's range and over long sums,
on the GPU against 64-bit references."""
import numpy as np
import pytest
import torch

from test_fp8_path import U16, U32, Y_REL, _bwd_ref, _check_fp8, _norm_ref, _np, _rand

pytestmark = pytest.mark.gpu

# a warp a row, a CTA a row, straight from memory, and the same with rows that start anywhere
WIDTHS = [264, 4096, 16392, 903, 1111, 20001]


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("size,weight", [(1e15, 1e25), (1e-17, 1e-25)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_whose_products_leave_the_range(cuda_lib, cols, size, weight, dtype):
    """h * weight lies outside of fp32's normal numbers, y = h rstd weight
    well inside."""
    x = (_rand((7, cols), torch.float32, 1) * size).to(dtype)
    w = (1 + 0.1 * torch.randn(cols, device="cuda")) * weight
    got = cuda_lib.kda_rms_norm(x, w, eps=0.0, fp8=True)
    y = _norm_ref(_np(x), _np(w), 0.0)
    u = U16 if dtype == torch.bfloat16 else U32
    assert np.all(np.abs(_np(got.out) - y) <= np.abs(y) * (Y_REL + u * (1 + Y_REL)))
    _check_fp8(got.fp8, y, Y_REL)


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_bwd_of_small_rows(cuda_lib, cols, residual, dtype):
    """rstd is about 1e17 and its square beyond fp32, the gradients are well
    inside.  Sums of at most 70 serial roundings each, and a dozen more, as
    for ordinary rows; a column of dweight adds up to seven rows in lanes of
    their own."""
    h = (_rand((7, cols), torch.float32, 2) * 1e-17).to(dtype)
    g = (_rand((7, cols), torch.float32, 3) * 1e9).to(dtype)
    d = (_rand((7, cols), torch.float32, 4) * 1e26).to(dtype) if residual else None
    w = 1 + 0.1 * torch.randn(cols, device="cuda")
    dx, dw = cuda_lib.kda_rms_norm_bwd(g, h, w, d, eps=0.0)
    want, want_w, mag, mag_w = _bwd_ref(_np(g), _np(h), _np(w), _np(d) if residual else 0.0, 0.0)
    tol = mag * (2 * 70 + 12) * U32 + (np.abs(want) * U16 if dtype == torch.bfloat16 else 0)
    assert np.all(np.abs(_np(dx) - want) <= tol)
    assert np.all(np.abs(_np(dw) - want_w) <= mag_w * (7 + 45) * U32)


def _positive_products(cuda_lib, m, n, k, seed):
    """Operands of a "tn" product whose terms are all positive, and the
    product in 64 bits, worked out on the GPU in pieces of k."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    a, b = (cuda_lib.kda_fp8_quantize(torch.randn(k, c, device="cuda", generator=g).abs(), "col")[0] for c in (m, n))
    want = torch.zeros(m, n, dtype=torch.float64, device="cuda")
    step = 1 << 18  # whole words of scales: 512 rows each
    for i in range(0, k, step):
        part = []
        for x in (a, b):
            rows = x.data[i:i + step].double()
            e = x.scales.view(torch.uint8)[i // 512:-(-(i + len(rows)) // 512)].double() - 127
            part.append(rows * torch.exp2(e).permute(0, 2, 1).flatten(0, 1).repeat_interleave(128, 0)[:len(rows)])
        want += part[0].t() @ part[1]
    return a, b, want


def test_bf16_products_of_a_very_long_sum(cuda_lib):
    """Four million positive terms.  A step of 32 terms may drop 2^-23 of the
    running sum, and a span holds 4,096 steps, over which the sum grows from
    nothing: half of 4096 * 2^-23 at most.  Sums of 128 spans in fp32 add at
    most 128 * 2^-24.  The rounding to bf16 is monotone: the result lies
    between the two bounds as they round."""
    a, b, want = _positive_products(cuda_lib, 16, 128, (1 << 22) + 100, 5)
    rel = 0.5 * 4096 * 2.0 ** -23 + 128 * 2.0 ** -24
    got = cuda_lib.kda_fp8_matmul(a, b, "tn")
    assert bool((got >= (want * (1 - rel)).bfloat16()).all() and (got <= (want * (1 + rel)).bfloat16()).all())
    assert cuda_lib.kda_fp8_matmul_status() == cuda_lib.KDA_OK


@pytest.mark.parametrize("m,n", [(3, 200), (300, 1000), (1000, 4104), (1001, 4099)])
@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
def test_bf16_products_in_several_spans_are_exact(cuda_lib, form, m, n):
    """A k just past one span (few rows, single CTAs, pairs of CTAs, odd
    sizes): entries of -1, 0 and 1 have sums that fp32 holds exactly, so the
    result is the exact one rounded to bf16."""
    k = 132_000
    g = torch.Generator(device="cuda").manual_seed(6)
    make = lambda *s: torch.randint(-1, 2, s, device="cuda", generator=g, dtype=torch.int8).bfloat16()  # noqa: E731
    sa, sb = {"nt": ((m, k), (n, k)), "nn": ((m, k), (k, n)), "tn": ((k, m), (k, n))}[form]
    x, y = make(*sa), make(*sb)
    a, = cuda_lib.kda_fp8_quantize(x, "col" if form == "tn" else "row")
    b, = cuda_lib.kda_fp8_quantize(y, "col" if form == "tn" else "tile")
    got = cuda_lib.kda_fp8_matmul(a, b, form)
    want = torch.zeros(m, n, dtype=torch.float64, device="cuda")
    for i in range(0, k, 1 << 14):
        s = slice(i, i + (1 << 14))
        A = x[s].t() if form == "tn" else x[:, s]
        B = y[:, s].t() if form == "nt" else y[s]
        want += A.double() @ B.double()
    assert torch.equal(got, want.bfloat16())
    assert torch.equal(cuda_lib.kda_fp8_matmul(a, b, form, out_dtype=torch.float32).double(), want)


@pytest.mark.parametrize("m,n", [(3, 130), (640, 1300), (4096, 2048)])
@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
def test_fp32_products_lose_little_beside_a_large_term(cuda_lib, form, m, n):
    """One term of 2^26, then 32 terms at a time that add up to 1.5: beside
    the large one a step may lose its 1.5, but not beyond the span of k that
    the large one is in, 48 steps at most.  The sums of the six spans round to
    multiples of 8."""
    k = 8192
    a, b = torch.ones(m, k, device="cuda"), torch.full((k, n), 1.5 / 32, device="cuda")
    a[:, :128], b[:128] = 0, 0
    a[:, 5], b[5] = 2.0 ** 13, 2.0 ** 13
    want = 2.0 ** 26 + 1.5 * (k - 128) / 32
    x = a.t().contiguous() if form == "tn" else a
    y = b.t().contiguous() if form == "nt" else b
    x8, = cuda_lib.kda_fp8_quantize(x, "col" if form == "tn" else "row")
    y8, = cuda_lib.kda_fp8_quantize(y, "col" if form == "tn" else "tile")
    got = cuda_lib.kda_fp8_matmul(x8, y8, form, out_dtype=torch.float32).double()
    assert float((got - want).abs().max()) <= 48 * 1.5 + 6 * 4
