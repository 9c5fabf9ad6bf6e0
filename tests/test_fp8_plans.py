"""The matrix product of scaled 8-bit matrices in every tile width, output
path and number of spans that its plan gives large problems, and the norm's
and the binding's less common ways, on the GPU."""
import ctypes

import numpy as np
import pytest
import torch

import fp8_testutil as ref
from test_fp8_path import NORM_SHAPES, U32, _bwd_ref, _np, _operands, _product, _rand

pytestmark = pytest.mark.gpu

# Pairs of CTAs in tiles of 160, 192, 128 and 224 rows, each with rows of the
# result on 16 bytes and not.  k: three blocks; two spans of fp32 sums, the
# second one short; four.
PAIR_SHAPES = [(2900, 2048), (2901, 2047), (3500, 2048), (3501, 2047), (2200, 2048), (2201, 2047), (2500, 2600), (2501, 2599)]


def _integers(shape, seed):
    """Up to 4, times a power of two for each 128 x 128 block: sums are exact
    in fp32 whatever their order."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randint(-4, 5, shape, device="cuda", generator=g).float()
    e = torch.exp2(torch.randint(-1, 2, [ref.blocks(s) for s in shape], device="cuda", generator=g).float())
    return x * e.repeat_interleave(128, 0)[:shape[0]].repeat_interleave(128, 1)[:, :shape[1]]


def _exact(form, a, b):
    return _product(form, *(torch.from_numpy(ref.values(x)).cuda() for x in (a, b)))


@pytest.mark.parametrize("k", [272, 1736, 5000])
@pytest.mark.parametrize("m,n", PAIR_SHAPES)
@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
def test_pairs_in_every_width_are_exact(cuda_lib, form, m, n, k):
    a, b = _operands(cuda_lib, form, m, n, k, 200, _integers)
    want = _exact(form, a, b)
    assert torch.equal(cuda_lib.kda_fp8_matmul(a, b, form, out_dtype=torch.float32).double(), want)
    assert torch.equal(cuda_lib.kda_fp8_matmul(a, b, form), want.bfloat16())
    assert cuda_lib.kda_fp8_matmul_status() == cuda_lib.KDA_OK


@pytest.mark.parametrize("left,pitch", [(5, 2063), (8, 2072)])
@pytest.mark.parametrize("m", [2201, 2901, 3501])
@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
def test_pairs_write_only_their_result(cuda_lib, form, m, left, pitch):
    """Into the middle of a wider buffer, from an odd column on and from one
    that TMA stores take: nothing around the result is touched."""
    n, k = 2047, 1736
    a, b = _operands(cuda_lib, form, m, n, k, 210, _integers)
    want = _exact(form, a, b)
    for dtype in (torch.float32, torch.bfloat16):
        buf = torch.full((m + 6, pitch), 7.0, dtype=dtype, device="cuda")
        out = buf[3:3 + m, left:left + n]
        cuda_lib.kda_fp8_matmul(a, b, form, out=out)
        assert torch.equal(out, want.to(dtype))
        out.fill_(7.0)
        assert torch.all(buf == 7.0)


@pytest.mark.parametrize("m,n,k", [(1, 130, 4096), (5, 1000, 8200), (33, 257, 2064), (64, 129, 8192)])
@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
def test_split_products_write_only_their_result(cuda_lib, form, m, n, k):
    """The same where k is split over a cluster."""
    a, b = _operands(cuda_lib, form, m, n, k, 260, _integers)
    want = _exact(form, a, b)
    for dtype in (torch.float32, torch.bfloat16):
        for left in (5, 8):
            buf = torch.full((m + 6, n + 16), 7.0, dtype=dtype, device="cuda")
            out = buf[3:3 + m, left:left + n]
            cuda_lib.kda_fp8_matmul(a, b, form, out=out)
            assert torch.equal(out, want.to(dtype))
            out.fill_(7.0)
            assert torch.all(buf == 7.0)


@pytest.mark.parametrize("m,n,k", [(3, 130, 1100), (300, 200, 300), (2201, 2047, 300)])
@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
def test_scales_at_both_ends(cuda_lib, form, m, n, k):
    """One operand about 2^-121, with scale bytes down to 0, the other about
    2^122: the products are of ordinary size and exact."""
    a, b = _operands(cuda_lib, form, m, n, k, 270,
                     lambda s, seed: _integers(s, seed) * (2.0 ** -121 if seed == 270 else 2.0 ** 122))
    assert int(a.scales.view(torch.uint8).min()) == 0
    want = _exact(form, a, b)
    assert float(want.abs().max()) > 1
    assert torch.equal(cuda_lib.kda_fp8_matmul(a, b, form, out_dtype=torch.float32).double(), want)


@pytest.mark.parametrize("m,n", [(70, 200), (2201, 2047)])
def test_scale_that_is_nan(cuda_lib, m, n):
    """Byte 255 stands for NaN: it reaches the results of its row, or of its
    tile's columns, and no others."""
    k = 700
    a, b = _operands(cuda_lib, "nt", m, n, k, 280, _integers)
    want = _exact("nt", a, b)
    a.scales.view(torch.uint8)[1, 17, 0] = 255       # row 17, columns 512 to 639
    b.scales.view(torch.uint8)[1, 2] = 255           # rows 128 and on, columns 256 to 383
    got = cuda_lib.kda_fp8_matmul(a, b, out_dtype=torch.float32).double()
    bad = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    bad[17], bad[:, 128:256] = True, True
    assert torch.equal(torch.isnan(got), bad)
    assert torch.equal(got[~bad], want[~bad])


def test_products_and_layers_on_several_streams(cuda_lib):
    """Products of both kernels, norms, quantisers and the chunked forward at
    once on streams of their own, whose kernels share SMs and tensor memory:
    the results are those of each alone."""
    g = torch.Generator(device="cuda").manual_seed(290)
    q, k, v = (torch.randn(2, 512, 8, 128, device="cuda", generator=g).bfloat16() for _ in range(3))
    gate, beta = -torch.rand(2, 512, 8, 128, device="cuda", generator=g), torch.rand(2, 512, 8, device="cuda", generator=g)
    large = _operands(cuda_lib, "nt", 2500, 2600, 1024, 291, _integers)
    few = _operands(cuda_lib, "nt", 3, 2048, 4096, 293, _integers)
    some = _operands(cuda_lib, "tn", 300, 1000, 2000, 295, _integers)
    x = _rand((3000, 2048), torch.bfloat16, 297)
    calls = [lambda: cuda_lib.kda_fp8_matmul(*large), lambda: cuda_lib.kda_fp8_matmul(*few),
             lambda: cuda_lib.kda_fp8_matmul(*some, "tn", out_dtype=torch.float32),
             lambda: cuda_lib.kda_chunk_fwd(q, k, v, gate, beta)[0], lambda: cuda_lib.kda_rms_norm(x, None, x).out,
             lambda: cuda_lib.kda_fp8_quantize(x, ("row", "col"))[1].data.view(torch.uint8)]
    want = [f() for f in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(20):
        got = []
        for f, s in zip(calls, streams):
            with torch.cuda.stream(s):
                for _ in range(3):
                    out = f()
                got.append(out)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert cuda_lib.kda_fp8_matmul_status() == cuda_lib.KDA_OK


@pytest.mark.parametrize("rows,cols", NORM_SHAPES + [(700, 256), (1300, 100)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_bwd_weight_gradient(cuda_lib, rows, cols, dtype):
    """A column of dweight adds rows / 608 in a thread, up to 1,216 partial
    rows over 64 lanes (19 each), the lanes of a warp that share it (two
    exchanges) and 16 warps; up to eight warps before that; 45 in n itself."""
    h, g = _rand((rows, cols), dtype, 7), _rand((rows, cols), dtype, 8)
    w = 1 + 0.1 * torch.randn(cols, device="cuda")
    _, dw = cuda_lib.kda_rms_norm_bwd(g, h, w, eps=1e-6)
    _, want, _, mag = _bwd_ref(_np(g), _np(h), _np(w), 0.0, float(np.float32(1e-6)))
    assert np.all(np.abs(_np(dw) - want) <= mag * (rows / 608 + 1 + 19 + 2 + 16 + 8 + 45) * U32 + 1e-38)


@pytest.mark.parametrize("cols", [264, 1111, 4096])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_residual_sums_at_the_ends_of_the_range(cuda_lib, cols, dtype):
    """The stream's addition rounds once, also among the smallest numbers,
    with zeros of either sign, infinities and NaN."""
    x, r = (_rand((9, cols), torch.float32, s) for s in (220, 221))
    x[0] *= 1e-38
    r[0] *= 1e-38
    x[1], r[1] = x[1] * 1e-40, r[1] * 1e-42
    r[2] = -x[2]
    x[3], r[3] = 0.0, -0.0
    x[4], r[4] = -0.0, -0.0
    x[5, 3], r[5, 3], x[6, 4], x[7, 5] = float("inf"), float("-inf"), float("inf"), float("nan")
    x[8], r[8] = 3e38, 3e38
    x, r = x.to(dtype), r.to(dtype)
    got = cuda_lib.kda_rms_norm(x, None, r).residual_out
    want = (x.double() + r.double()).to(torch.float32).to(dtype) if dtype == torch.bfloat16 else x + r
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    fine = ~torch.isnan(want)
    bits = torch.int16 if dtype == torch.bfloat16 else torch.int32
    assert torch.equal(got.view(bits)[fine], want.view(bits)[fine])


def test_binding_without_the_short_allocator(cuda_lib, monkeypatch):
    """Where torch lacks the allocation that the binding prefers, its public
    one gives the same results."""
    x = _rand((300, 1000), torch.bfloat16, 230)

    def calls():
        n = cuda_lib.kda_rms_norm(x, None, x, fp8=True)
        w, = cuda_lib.kda_fp8_quantize(x, "tile")
        dx, dw = cuda_lib.kda_rms_norm_bwd(n.out, n.residual_out)
        y = cuda_lib.kda_fp8_matmul(n.fp8, w)
        return [n.out, n.residual_out, n.fp8.data.view(torch.uint8), n.fp8.scales.view(torch.uint8), dx, dw, y]

    want = calls()
    before = cuda_lib._alloc
    monkeypatch.setattr(cuda_lib, "_F8", None)
    monkeypatch.setattr(cuda_lib, "_alloc", before)  # put back afterwards
    monkeypatch.delattr(torch._C._dynamo.guards, "_empty_strided_cuda", raising=False)
    got = calls()
    assert cuda_lib._alloc is not before
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert [t.stride() for t in got] == [t.stride() for t in want]


@pytest.mark.parametrize("m,n", [(5, 130), (2201, 2047), (2901, 2048)])
@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
def test_operands_inside_of_wider_buffers(cuda_lib, form, m, n):
    """What stands beside an operand's rows is NaN: none of it is read into a
    sum, in either operand, also where a row ends inside of 16 bytes."""
    k = 1741
    a, b = _operands(cuda_lib, form, m, n, k, 240, _integers)
    want = _exact(form, a, b)

    def widened(x):
        rows, cols = x.data.shape
        buf = torch.full((rows + 2, (cols + 31) // 16 * 16), 0x7F, dtype=torch.uint8, device="cuda")
        buf[1:1 + rows, :cols] = x.data.view(torch.uint8)
        return cuda_lib.Fp8Matrix(buf.view(torch.float8_e4m3fn)[1:1 + rows, :cols], x.scales, x.kind)

    for dtype in (torch.float32, torch.bfloat16):
        assert torch.equal(cuda_lib.kda_fp8_matmul(widened(a), widened(b), form, out_dtype=dtype), want.to(dtype))


class _Guarded:
    """Device buffers between bands of 4,096 bytes of 0xA5."""

    def __init__(self):
        self.bands = []

    def new(self, nbytes):
        buf = torch.full((8192 + (nbytes + 15) // 16 * 16,), 0xA5, dtype=torch.uint8, device="cuda")
        self.bands.append((buf, nbytes))
        return buf[4096:4096 + nbytes]

    def intact(self):
        return all(bool((b[:4096] == 0xA5).all()) and bool((b[4096 + n:] == 0xA5).all()) for b, n in self.bands)


@pytest.mark.parametrize("rows,cols", NORM_SHAPES + [(20001, 903)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_and_quantiser_write_only_their_results(cuda_lib, rows, cols, dtype):
    """Guard bands around every output, and a pitch of the 8-bit values with
    room beside each row."""
    k, lib = cuda_lib, cuda_lib.load_library()
    code, es = (k.KDA_BF16, 2) if dtype == torch.bfloat16 else (k.KDA_F32, 4)
    x, r, g = (_rand((rows, cols), dtype, s) for s in (250, 251, 252))
    stream = torch.cuda.current_stream().cuda_stream
    ld = (cols + 15) // 16 * 16 + 32
    rb, cb = ref.blocks(rows), ref.blocks(cols)
    buf = _Guarded()

    def beside(q):
        """The bytes to the right of the values have not been written."""
        return bool((q.view(rows, ld)[:, cols:] == 0xA5).all())

    want = k.kda_rms_norm(x, None, r, fp8=True)
    h, out, q, s = buf.new(rows * cols * es), buf.new(rows * cols * es), buf.new(rows * ld), buf.new((cb + 3) // 4 * rows * 4)
    a = k.kda_rms_norm_args(rows, cols, code, x.data_ptr(), r.data_ptr(), None, 1e-6, h.data_ptr(), out.data_ptr(),
                            q.data_ptr(), ld, s.data_ptr())
    assert lib.kda_rms_norm(ctypes.byref(a), stream) == k.KDA_OK
    assert buf.intact() and beside(q)
    assert torch.equal(h.view(dtype).view(rows, cols), want.residual_out) and torch.equal(out.view(dtype).view(rows, cols), want.out)
    assert torch.equal(q.view(rows, ld)[:, :cols], want.fp8.data.view(torch.uint8))
    assert torch.equal(s, want.fp8.scales.view(torch.uint8).flatten())

    want_dx, want_dw = k.kda_rms_norm_bwd(g, x, None, r)
    need = lib.kda_rms_norm_bwd_workspace_size(rows, cols)
    dx, dw, ws = buf.new(rows * cols * es), buf.new(cols * 4), buf.new(need)
    a = k.kda_rms_norm_bwd_args(rows, cols, code, g.data_ptr(), x.data_ptr(), None, r.data_ptr(), 1e-6, dx.data_ptr(),
                                dw.data_ptr(), ws.data_ptr(), need)
    assert lib.kda_rms_norm_bwd(ctypes.byref(a), stream) == k.KDA_OK
    assert buf.intact()
    assert torch.equal(dx.view(dtype).view(rows, cols), want_dx) and torch.equal(dw.view(torch.float32), want_dw)

    kinds = ("row", "col", "tile")
    parts = k.kda_fp8_quantize(x, kinds)
    vals = [buf.new(rows * ld) for _ in kinds]
    scales = [buf.new((cb + 3) // 4 * rows * 4), buf.new((rb + 3) // 4 * cols * 4), buf.new(rb * cb)]
    a = k.kda_fp8_quantize_args(rows, cols, code, x.data_ptr(), ld, *(t.data_ptr() for t in vals), *(t.data_ptr() for t in scales))
    assert lib.kda_fp8_quantize(ctypes.byref(a), stream) == k.KDA_OK
    assert buf.intact()
    for p, v, e in zip(parts, vals, scales):
        assert beside(v) and torch.equal(v.view(rows, ld)[:, :cols], p.data.view(torch.uint8))
        assert torch.equal(e, p.scales.view(torch.uint8).flatten())
