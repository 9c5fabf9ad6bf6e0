"""Host-side checks of the 8-bit projection path, without a GPU: refusals of
the C calls and of the Python binding."""
import ctypes

import pytest
import torch

import chunked_kimi_delta_gb300 as kda
from chunked_kimi_delta_gb300 import build as kbuild

BASE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda.load_library()


def _fill(args, fields, /, **kw):
    for key, val in {**fields, **kw}.items():
        setattr(args, key, val)
    return args


def _norm(**kw):
    return _fill(kda.kda_rms_norm_args(), dict(rows=4, cols=256, dtype=kda.KDA_BF16, x=BASE, residual=2 * BASE,
                 weight=3 * BASE, eps=1e-6, residual_out=4 * BASE, out=5 * BASE, fp8=6 * BASE, ld_fp8=256,
                 fp8_scales=7 * BASE), **kw)


def _bwd(**kw):
    return _fill(kda.kda_rms_norm_bwd_args(), dict(rows=4, cols=256, dtype=kda.KDA_BF16, d_out=BASE, h=2 * BASE,
                 weight=3 * BASE, d_residual=4 * BASE, eps=1e-6, dx=5 * BASE, dweight=6 * BASE,
                 workspace=7 * BASE, workspace_bytes=4 * 256 * 4), **kw)


def _quant(**kw):
    return _fill(kda.kda_fp8_quantize_args(), dict(rows=4, cols=256, dtype=kda.KDA_F32, x=BASE, ld=256, row=2 * BASE,
                 row_scales=3 * BASE, col=4 * BASE, col_scales=5 * BASE, tile=6 * BASE, tile_scales=7 * BASE), **kw)


def _mm(**kw):
    return _fill(kda.kda_fp8_matmul_args(), dict(m=4, n=100, k=200, form=kda.KDA_FP8_NT, a=BASE, lda=208,
                 a_scales=2 * BASE, b=3 * BASE, ldb=208, b_scales=4 * BASE, out=5 * BASE, ldo=100,
                 out_dtype=kda.KDA_BF16, workspace=6 * BASE, workspace_bytes=256), **kw)


INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 1, 2, 3, 4


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), INVALID), (dict(cols=0), INVALID), (dict(x=None), INVALID), (dict(dtype=7), INVALID),
    (dict(out=None, fp8=None), INVALID), (dict(residual_out=None), INVALID),
    (dict(residual_out=5 * BASE), INVALID), (dict(fp8_scales=None), INVALID),
    (dict(ld_fp8=240), INVALID), (dict(cols=32769, ld_fp8=32784), UNSUPPORTED), (dict(rows=1 << 31), UNSUPPORTED),
    (dict(x=BASE + 2), ALIGNMENT), (dict(weight=BASE + 4), ALIGNMENT), (dict(ld_fp8=264), ALIGNMENT),
    (dict(fp8_scales=BASE + 8), ALIGNMENT), (dict(rows=0), 0)])
def test_norm_refusals(lib, kw, want):
    assert lib.kda_rms_norm(ctypes.byref(_norm(**kw)), None) == want
    assert lib.kda_rms_norm(None, None) == INVALID


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), INVALID), (dict(cols=0), INVALID), (dict(h=None), INVALID), (dict(d_out=None), INVALID),
    (dict(dx=None), INVALID), (dict(dtype=-1), INVALID), (dict(cols=40000), UNSUPPORTED),
    (dict(d_residual=BASE + 8), ALIGNMENT), (dict(workspace=None), WORKSPACE),
    (dict(workspace_bytes=4 * 256 * 4 - 1), WORKSPACE), (dict(workspace=BASE + 16), ALIGNMENT)])
def test_norm_bwd_refusals(lib, kw, want):
    assert lib.kda_rms_norm_bwd(ctypes.byref(_bwd(**kw)), None) == want
    assert lib.kda_rms_norm_bwd(None, None) == INVALID
    assert lib.kda_rms_norm_bwd_workspace_size(4, 256) == 4 * 256 * 4
    assert lib.kda_rms_norm_bwd_workspace_size(-1, 256) == 0
    assert lib.kda_rms_norm_bwd_workspace_size(4, 40000) == 0


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), INVALID), (dict(cols=-1), INVALID), (dict(x=None), INVALID),
    (dict(row=None, col=None, tile=None), INVALID), (dict(row_scales=None), INVALID),
    (dict(col_scales=None), INVALID), (dict(tile_scales=None), INVALID), (dict(ld=240), INVALID),
    (dict(ld=260), ALIGNMENT), (dict(x=BASE + 4), ALIGNMENT), (dict(col=BASE + 8), ALIGNMENT),
    (dict(rows=1 << 40, cols=1 << 20, ld=1 << 20), UNSUPPORTED), (dict(rows=1 << 37), UNSUPPORTED), (dict(rows=0), 0), (dict(cols=0), 0)])
def test_quantize_refusals(lib, kw, want):
    assert lib.kda_fp8_quantize(ctypes.byref(_quant(**kw)), None) == want
    assert lib.kda_fp8_quantize(None, None) == INVALID


@pytest.mark.parametrize("rows", [1 << 38, 1 << 46, 1 << 62, (1 << 63) - 1])
def test_quantize_refuses_any_number_of_blocks_past_its_limit(lib, rows):
    cols = (1 << 31) - 16
    assert lib.kda_fp8_quantize(ctypes.byref(_quant(rows=rows)), None) == UNSUPPORTED
    assert lib.kda_fp8_quantize(ctypes.byref(_quant(rows=rows, cols=cols, ld=cols)), None) == UNSUPPORTED


@pytest.mark.parametrize("kw,want", [
    (dict(m=-1), INVALID), (dict(n=-1), INVALID), (dict(k=-1), INVALID), (dict(form=3), INVALID),
    (dict(out_dtype=5), INVALID), (dict(flags=1), INVALID), (dict(a=None), INVALID), (dict(b_scales=None), INVALID), (dict(out=None), INVALID),
    (dict(ldo=99), INVALID), (dict(lda=192), INVALID), (dict(form=kda.KDA_FP8_NN, ldb=96), INVALID),
    (dict(form=kda.KDA_FP8_TN, lda=0), INVALID), (dict(lda=201), ALIGNMENT), (dict(ldb=216), ALIGNMENT),
    (dict(a=BASE + 8), ALIGNMENT), (dict(out=BASE + 1), ALIGNMENT), (dict(out_dtype=kda.KDA_F32, out=BASE + 2), ALIGNMENT),
    (dict(lda=1 << 31), UNSUPPORTED),
    (dict(m=(1 << 31) - 1), UNSUPPORTED), (dict(workspace=None), WORKSPACE), (dict(workspace_bytes=255), WORKSPACE),
    (dict(workspace=BASE + 128), ALIGNMENT), (dict(m=0), 0), (dict(n=0), 0)])
def test_matmul_refusals(lib, kw, want):
    assert lib.kda_fp8_matmul(ctypes.byref(_mm(**kw)), None) == want
    assert lib.kda_fp8_matmul(None, None) == INVALID


def test_binding_refusals(lib):
    x = torch.zeros(4, 256)
    with pytest.raises(ValueError, match="CUDA tensors"):
        kda.kda_rms_norm(x)
    with pytest.raises(ValueError, match="CUDA tensors"):
        kda.kda_fp8_quantize(x)
    with pytest.raises(ValueError, match="CUDA tensors"):
        kda.kda_rms_norm_bwd(x, x)
    with pytest.raises(ValueError, match="no result"):
        kda.kda_rms_norm(x, out=False)
    with pytest.raises(ValueError, match="weight"):
        kda.kda_rms_norm(x, torch.ones(255))
    with pytest.raises(ValueError, match="weight"):
        kda.kda_rms_norm(x, torch.ones(256, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="residual must"):
        kda.kda_rms_norm(x, None, torch.zeros(4, 255))
    with pytest.raises(ValueError, match="residual_out needs"):
        kda.kda_rms_norm(x, residual_out=x)
    with pytest.raises(ValueError, match="contiguous"):
        kda.kda_rms_norm(torch.zeros(256, 4).t())
    with pytest.raises(ValueError, match="d_out must"):
        kda.kda_rms_norm_bwd(x[:3], x)
    with pytest.raises(ValueError, match="each once"):
        kda.kda_fp8_quantize(x, kinds=("row", "row"))
    with pytest.raises(ValueError, match="each once"):
        kda.kda_fp8_quantize(x, kinds=("block",))
    with pytest.raises(ValueError, match="rows, cols"):
        kda.kda_fp8_quantize(x[0])


def _matrix(rows, cols, kind):
    data = torch.zeros(rows, -(-cols // 16) * 16, dtype=torch.uint8).view(torch.float8_e4m3fn)[:, :cols]
    return kda.Fp8Matrix(data, torch.zeros(kda._scale_shape(rows, cols, kind), dtype=torch.uint8).view(torch.float8_e8m0fnu), kind)


def test_binding_matmul_refusals(lib):
    a, b = _matrix(4, 256, "row"), _matrix(100, 256, "tile")
    with pytest.raises(ValueError, match="CUDA tensors"):
        kda.kda_fp8_matmul(a, b)
    with pytest.raises(ValueError, match="form"):
        kda.kda_fp8_matmul(a, b, "tt")
    with pytest.raises(ValueError, match="needs row scales"):
        kda.kda_fp8_matmul(_matrix(4, 256, "col"), b)
    with pytest.raises(ValueError, match="sum over"):
        kda.kda_fp8_matmul(a, b, "nn")
    with pytest.raises(TypeError, match="float8"):
        kda.kda_fp8_matmul(kda.Fp8Matrix(a.data.view(torch.uint8), a.scales, "row"), b)
    with pytest.raises(ValueError, match="have shape"):
        kda.kda_fp8_matmul(kda.Fp8Matrix(a.data, a.scales[:0], "row"), b)
    with pytest.raises(ValueError, match="out must"):
        kda.kda_fp8_matmul(a, b, out=torch.empty(4, 99))
    with pytest.raises(TypeError, match="unsupported dtype"):
        kda.kda_fp8_matmul(a, b, out=torch.empty(4, 100, dtype=torch.float16))
    with pytest.raises(ValueError, match="dense rows"):
        kda.kda_fp8_matmul(a, b, out=torch.empty(100, 4).t())
