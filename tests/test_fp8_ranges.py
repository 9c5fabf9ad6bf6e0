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
