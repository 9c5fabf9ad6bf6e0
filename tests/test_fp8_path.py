"""The 8-bit projection path on the GPU against 64-bit references: RMS norm
(forward, backward), quantiser, matrix product."""
import numpy as np
import pytest
import torch

import fp8_testutil as ref

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24   # unit roundoff of fp32
U16 = 2.0 ** -8    # unit roundoff of bf16 (8 significant bits)
# y = h * rstd * w: the sum of squares passes through at most 32 serial additions in a
# thread, 5 shuffles and 32 warps, whose relative error halves in the root; division,
# addition of eps, root, reciprocal and two products add at most 6 roundings.
Y_REL = (35 + 6) * U32


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(*shape, device="cuda", generator=g) * scale
    x *= torch.exp(torch.randn(shape[0], 1, device="cuda", generator=g))
    return x.to(dtype)


def _norm_ref(h, w, eps):
    return h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * w


def _check_fp8(m, y, rel):
    """m stands for y, whose elements are known to a relative error rel."""
    kind = m.kind
    amax = ref.block_amax(y, kind)
    e = m.scales.view(torch.uint8).cpu().numpy().astype(np.int64)
    lo, hi = ref.scale_exponent(amax * (1 - rel)), ref.scale_exponent(amax * (1 + rel))
    slo, shi = ref.stored_scales(lo, kind), ref.stored_scales(hi, kind)
    assert np.all((e == slo) | (e == shi)), "block exponents"
    s = np.ldexp(1.0, ref.expand(hi, kind, *y.shape))
    # half a step of e4m3 (2^-4 of the value, 2^-10 of the scale near zero)
    tol = np.maximum(np.abs(y) * 2.0 ** -4, s * 2.0 ** -10) * (1 + 2 * rel) + np.abs(y) * rel
    assert np.all(np.abs(ref.values(m) - y) <= tol), "e4m3 values"


NORM_SHAPES = [(1, 1), (3, 7), (2, 128), (5, 130), (1, 4096), (33, 512), (17, 1111), (4, 2048),
               (7, 4100), (2, 5000), (3, 16392), (2, 32768), (2, 32767), (8001, 264), (4003, 1023)]


@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("residual", [False, True])
def test_norm(cuda_lib, rows, cols, dtype, residual):
    x, r = _rand((rows, cols), dtype, 1), _rand((rows, cols), dtype, 2) if residual else None
    w = 1 + 0.1 * torch.randn(cols, device="cuda")
    got = cuda_lib.kda_rms_norm(x, w, r, eps=1e-6, fp8=True)
    h = x
    if residual:
        h = (x.float() + r.float()).to(dtype)
        assert torch.equal(got.residual_out, h)
    else:
        assert got.residual_out is None
    y = _norm_ref(_np(h), _np(w), float(np.float32(1e-6)))
    u = U16 if dtype == torch.bfloat16 else U32
    assert np.all(np.abs(_np(got.out) - y) <= np.abs(y) * (Y_REL + u * (1 + Y_REL)) + 1e-38)
    _check_fp8(got.fp8, y, Y_REL)
    alone = cuda_lib.kda_rms_norm(x, w, r, eps=1e-6, fp8=True, out=False)
    assert alone.out is None
    assert torch.equal(alone.fp8.data.view(torch.uint8), got.fp8.data.view(torch.uint8))
    assert torch.equal(alone.fp8.scales.view(torch.uint8), got.fp8.scales.view(torch.uint8))


def test_norm_without_weight_in_place_and_zero_rows(cuda_lib):
    x, r = _rand((9, 384), torch.bfloat16, 3), _rand((9, 384), torch.bfloat16, 4)
    want = cuda_lib.kda_rms_norm(x, None, r)
    ones = cuda_lib.kda_rms_norm(x, torch.ones(384, device="cuda"), r)
    assert torch.equal(want.out, ones.out)
    x2, r2 = x.clone(), r.clone()
    got = cuda_lib.kda_rms_norm(x2, None, r2, residual_out=r2, out=x2)
    assert got.out is x2 and got.residual_out is r2
    assert torch.equal(x2, want.out) and torch.equal(r2, want.residual_out)
    empty = cuda_lib.kda_rms_norm(x[:0], None, r[:0], fp8=True)
    assert empty.out.shape == (0, 384) and empty.fp8.data.shape == (0, 384)
    # a row of zeros: zeros, scale one
    z = cuda_lib.kda_rms_norm(torch.zeros(2, 256, device="cuda"), fp8=True)
    assert float(z.out.abs().max()) == 0 and float(z.fp8.data.float().abs().max()) == 0
    assert torch.all(z.fp8.scales.view(torch.uint8) == 127)


def test_norm_nan_and_inf_stay_in_their_row(cuda_lib):
    x = _rand((4, 300), torch.float32, 5)
    clean = cuda_lib.kda_rms_norm(x, fp8=True)
    x[1, 17], x[2, 5] = float("nan"), float("inf")
    got = cuda_lib.kda_rms_norm(x, fp8=True)
    for r in (0, 3):
        assert torch.equal(got.out[r], clean.out[r])
        assert torch.equal(got.fp8.data[r].view(torch.uint8), clean.fp8.data[r].view(torch.uint8))
    assert torch.all(torch.isnan(got.out[1]))
    # an infinite sum of squares: rstd is 0, finite elements become 0, the infinity NaN
    assert torch.isnan(got.out[2, 5]) and torch.isnan(got.fp8.data[2, 5].float())
    assert float(torch.nan_to_num(got.out[2]).abs().max()) == 0


@pytest.mark.parametrize("cols", [256, 200, 4096, 1111])
@pytest.mark.parametrize("size", [1e-34, 1e-37, 1e-39])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_of_tiny_values(cuda_lib, cols, size, dtype):
    """Values near the lower end of fp32, with zeros among them: y * 2^-e is
    of ordinary size, the factors that lead there are not."""
    x = (_rand((5, cols), torch.float32, 31) * size).to(dtype)
    x[1, ::3] = 0
    x[2, :128] = 0
    got = cuda_lib.kda_rms_norm(x, fp8=True)
    y = x.double().cpu().numpy() / np.sqrt(1e-6)
    # e4m3 keeps 4 bits (half a step: 2^-4 of the value) and, below its normal
    # range, steps of 2^-9 of the scale (448 * 2^e < 2 max |y|, e >= -127);
    # fp32 adds 2^-20 and its own smallest step
    amax = np.abs(y).max()
    tol = np.abs(y) * (2.0**-4 + 2.0**-20) + max(2 * amax / 448, 2.0**-127) * 2.0**-10 + 2.0**-147
    assert np.all(np.abs(ref.values(got.fp8) - y) <= tol)


def test_norm_leading_dims_and_another_stream(cuda_lib):
    x = _rand((6 * 5, 640), torch.bfloat16, 6).view(6, 5, 640)
    want = cuda_lib.kda_rms_norm(x.view(30, 640), fp8=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = cuda_lib.kda_rms_norm(x, fp8=True, stream=side)
    side.synchronize()
    assert got.out.shape == x.shape and torch.equal(got.out.view(30, 640), want.out)
    assert torch.equal(got.fp8.data.view(torch.uint8), want.fp8.data.view(torch.uint8))


@pytest.mark.parametrize("handle", [False, True])
def test_results_and_scratch_belong_to_the_stream_of_the_call(cuda_lib, handle):
    """Memory of a call on another stream is not handed out again by the
    current one: the scratch of the backward is let go of before the call runs."""
    k = cuda_lib
    x = _rand((300, 1000), torch.bfloat16, 8)
    want_dx, want_dw = k.kda_rms_norm_bwd(x, x)
    aq, wq = k.kda_fp8_quantize(x, ("row", "tile"))
    want_y = k.kda_fp8_matmul(aq, wq, "nt")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    stream = side.cuda_stream if handle else side
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # about 10 ms: what follows on `side` has not run yet
    y = k.kda_fp8_matmul(aq, wq, "nt", stream=stream)
    q, = k.kda_fp8_quantize(x, "row", stream=stream)
    dx, dw = k.kda_rms_norm_bwd(x, x, stream=stream)
    parts = k._ready().kda_rms_norm_bwd_workspace_size(300, 1000)
    scribble = [torch.full((parts // 4,), 7.0, device="cuda") for _ in range(4)]
    side.synchronize()
    torch.cuda.synchronize()
    assert all(bool((s == 7.0).all()) for s in scribble)
    assert torch.equal(dx, want_dx) and torch.equal(dw, want_dw) and torch.equal(y, want_y)
    assert torch.equal(q.data.view(torch.uint8), aq.data.view(torch.uint8))


def _bwd_ref(g, h, w, d, eps):
    """dx, dweight and, for the tolerances, the same sums over magnitudes."""
    rstd = 1 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    n = h * rstd
    gw = g * w
    dx = rstd * (gw - n * (gw * n).mean(-1, keepdims=True)) + d
    mag = rstd * (np.abs(gw) + np.abs(n) * np.abs(gw * n).mean(-1, keepdims=True)) + np.abs(d)
    return dx, (g * n).sum(0), mag, np.abs(g * n).sum(0)


@pytest.mark.parametrize("rows,cols", NORM_SHAPES + [(700, 256), (1300, 100)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_bwd(cuda_lib, rows, cols, dtype, residual):
    h, g = _rand((rows, cols), dtype, 7), _rand((rows, cols), dtype, 8)
    d = _rand((rows, cols), dtype, 9) if residual else None
    w = 1 + 0.1 * torch.randn(cols, device="cuda")
    dx, dw = cuda_lib.kda_rms_norm_bwd(g, h, w, d, eps=1e-6)
    want, want_w, mag, mag_w = _bwd_ref(_np(g), _np(h), _np(w), _np(d) if residual else 0.0, float(np.float32(1e-6)))
    # two sums of at most 70 serial roundings each, and a dozen more
    tol = mag * (2 * 70 + 12) * U32 + (np.abs(want) * U16 if dtype == torch.bfloat16 else 0)
    assert np.all(np.abs(_np(dx) - want) <= tol + 1e-38)
    # a column: rows / 608 in a thread, 76 partial rows in a lane, 8 lanes; Y_REL in n
    tol_w = mag_w * (rows / 608 + 1 + 76 + 8 + 45) * U32
    assert np.all(np.abs(_np(dw) - want_w) <= tol_w + 1e-38)
    again, dw2 = cuda_lib.kda_rms_norm_bwd(g, h, w, d, eps=1e-6)
    assert torch.equal(dx, again) and torch.equal(dw, dw2), "deterministic"
    only, none = cuda_lib.kda_rms_norm_bwd(g, h, w, d, eps=1e-6, want_dweight=False)
    assert none is None and torch.equal(only, dx)


def test_norm_bwd_against_differences(cuda_lib):
    """<d_out, y(h + t p)> by central differences of the 64-bit formula, along
    random directions in h and in the weight."""
    rows, cols = 11, 200
    h, g = _rand((rows, cols), torch.float32, 10), _rand((rows, cols), torch.float32, 11)
    w = 1 + 0.1 * torch.randn(cols, device="cuda")
    dx, dw = cuda_lib.kda_rms_norm_bwd(g, h, w, eps=1e-6)
    H, G, W = _np(h), _np(g), _np(w)
    rng = np.random.default_rng(0)
    f = lambda hh, ww: float((G * _norm_ref(hh, ww, float(np.float32(1e-6)))).sum())  # noqa: E731
    for _ in range(4):
        p, q, t = rng.standard_normal(H.shape) * np.abs(H), rng.standard_normal(cols), 1e-5
        dh = (f(H + t * p, W) - f(H - t * p, W)) / (2 * t)
        dq = (f(H, W + t * q) - f(H, W - t * q)) / (2 * t)
        # truncation t^2 and cancellation 1e-16 / t of sums of size |G| |y|, and fp32 in dx, dw
        size = np.abs(G * _norm_ref(H, W, 1e-6)).sum() * 10
        assert abs((_np(dx) * p).sum() - dh) <= 1e-5 * size
        assert abs((_np(dw) * q).sum() - dq) <= 1e-5 * size


def test_norm_bwd_in_place_and_zero_rows(cuda_lib):
    h, g, d = (_rand((8, 512), torch.bfloat16, s) for s in (12, 13, 14))
    want, _ = cuda_lib.kda_rms_norm_bwd(g, h, None, d)
    for i in range(3):
        t = [g.clone(), h.clone(), d.clone()]
        got, _ = cuda_lib.kda_rms_norm_bwd(t[0], t[1], None, t[2], dx=t[i])
        assert got is t[i] and torch.equal(got, want)
    dx, dw = cuda_lib.kda_rms_norm_bwd(g[:0], h[:0])
    assert dx.shape == (0, 512) and float(dw.abs().max()) == 0


QUANT_SHAPES = [(1, 1), (1, 128), (127, 129), (128, 128), (130, 77), (300, 1000), (513, 515), (5, 4104),
                (1030, 520)]


@pytest.mark.parametrize("rows,cols", QUANT_SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_bits(cuda_lib, rows, cols, dtype):
    x = _rand((rows, cols), dtype, 20)
    x[rows // 2] = 0
    x[:, cols // 2] *= 1e-30
    parts = cuda_lib.kda_fp8_quantize(x, kinds=("row", "col", "tile"))
    for p, kind in zip(parts, ("row", "col", "tile")):
        v, e = ref.quantize(_np(x), kind)
        assert p.kind == kind
        assert np.array_equal(p.scales.view(torch.uint8).cpu().numpy(), ref.stored_scales(e, kind)), kind
        assert np.array_equal(_np(p.data), v), kind
        alone, = cuda_lib.kda_fp8_quantize(x, kinds=kind)
        assert torch.equal(alone.data.view(torch.uint8), p.data.view(torch.uint8))
        assert torch.equal(alone.scales.view(torch.uint8), p.scales.view(torch.uint8))


def test_quantize_extremes(cuda_lib):
    """Exponents at both ends, exact powers around the rule's boundary, NaN and infinities."""
    x = torch.zeros(10, 256, device="cuda")
    x[0, 0], x[1, 0], x[2, 0] = 448.0, float(np.nextafter(np.float32(448), np.float32(500))), 3.4028234e38
    x[3, 0], x[4, 0], x[5, :3] = 1e-45, 1.17549435e-38, torch.tensor([1.0, float("nan"), 0.3])
    x[6, :3] = torch.tensor([float("inf"), -2.0, float("-inf")])
    x[7, :] = float("nan")
    x[8, :4] = torch.tensor([17.0, 19.0, -17.0, 448.0])   # ties between e4m3 neighbours
    x[9, :2] = torch.tensor([2.0 ** -10, 448.0])          # a tie with zero
    for kind in ("row", "col", "tile"):
        p, = cuda_lib.kda_fp8_quantize(x, kinds=kind)
        v, e = ref.quantize(_np(x), kind)
        assert np.array_equal(p.scales.view(torch.uint8).cpu().numpy(), ref.stored_scales(e, kind)), kind
        assert np.array_equal(_np(p.data), v, equal_nan=True), kind
    empty, = cuda_lib.kda_fp8_quantize(x[:0])
    assert empty.data.shape == (0, 256)


FORMS = {"nt": ("row", "tile"), "nn": ("row", "tile"), "tn": ("col", "col")}


def _operands(lib, form, m, n, k, seed, make):
    sa, sb = {"nt": ((m, k), (n, k)), "nn": ((m, k), (k, n)), "tn": ((k, m), (k, n))}[form]
    a, = lib.kda_fp8_quantize(make(sa, seed), kinds=FORMS[form][0])
    b, = lib.kda_fp8_quantize(make(sb, seed + 1), kinds=FORMS[form][1])
    return a, b


def _product(form, a, b):
    if form == "nt":
        return a @ b.T
    return a @ b if form == "nn" else a.T @ b


# m x n x k: single tokens, one tile and its neighbours, odd sizes, blocks of k that fill a
# scale word or not, long sums over few outputs, and one with several tiles in flight per SM
MM_SHAPES = [(1, 1, 1), (1, 256, 512), (2, 130, 100), (16, 128, 128), (17, 129, 129), (64, 384, 640),
             (100, 200, 300), (128, 128, 1024), (255, 257, 520), (300, 1111, 2064), (5, 4100, 384),
             (1000, 136, 1288), (9, 100, 8200), (2500, 2600, 272),
             # sums long enough to be taken out of tensor memory in between: k split or not, and pairs
             (3, 130, 34000), (640, 1300, 4200), (2500, 2600, 8400)]


@pytest.mark.parametrize("m,n,k", MM_SHAPES)
@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
def test_matmul(cuda_lib, form, m, n, k):
    a, b = _operands(cuda_lib, form, m, n, k, 30, lambda s, seed: _rand(s, torch.float32, seed))
    A, B = ref.values(a), ref.values(b)
    want, mag = _product(form, A, B), _product(form, np.abs(A), np.abs(B))
    # a 32-term step may drop one unit of the running sum's last place, and one in aligning its terms
    acc = mag * (k / 32 + 4) * 2 * 2.0 ** -23
    got = cuda_lib.kda_fp8_matmul(a, b, form, out_dtype=torch.float32)
    assert np.all(np.abs(_np(got) - want) <= acc + 1e-38)
    assert np.linalg.norm(_np(got) - want) <= 1e-5 * np.linalg.norm(want)
    half = cuda_lib.kda_fp8_matmul(a, b, form)
    assert half.dtype == torch.bfloat16
    assert np.all(np.abs(_np(half) - want) <= acc + (np.abs(want) + acc) * U16 + 1e-38)
    assert torch.equal(got, cuda_lib.kda_fp8_matmul(a, b, form, out_dtype=torch.float32)), "deterministic"
    assert cuda_lib.kda_fp8_matmul_status() == cuda_lib.KDA_OK


@pytest.mark.parametrize("m,n,k", MM_SHAPES)
@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
def test_matmul_of_small_integers_is_exact(cuda_lib, form, m, n, k):
    """Integers up to 4 with a block scale of 1, 2 or 4 times a power of two:
    every sum is a multiple of the smallest product below 2^24 of them, so
    fp32 holds it exactly whatever the order."""
    def make(shape, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x = torch.randint(-4, 5, shape, device="cuda", generator=g).float()
        # a power of two for each 128 x 128 block: every kind of block sees one exponent
        rb, cb = ref.blocks(shape[0]), ref.blocks(shape[1])
        e = torch.exp2(torch.randint(-1, 2, (rb, cb), device="cuda", generator=g).float())
        return x * e.repeat_interleave(128, 0)[:shape[0]].repeat_interleave(128, 1)[:, :shape[1]]
    a, b = _operands(cuda_lib, form, m, n, k, 40, make)
    want = _product(form, ref.values(a), ref.values(b))
    got = cuda_lib.kda_fp8_matmul(a, b, form, out_dtype=torch.float32)
    assert np.array_equal(_np(got), want)


@pytest.mark.parametrize("m,n,k", [(1, 20000, 200), (33, 19500, 136), (64, 39000, 264), (65, 19500, 136), (7, 40001, 4200)])
@pytest.mark.parametrize("form", ["nt", "nn"])
def test_matmul_of_few_rows_and_many_columns(cuda_lib, form, m, n, k):
    """A few tokens through a wide projection."""
    test_matmul(cuda_lib, form, m, n, k)


def test_matmul_pitches_streams_and_canaries(cuda_lib):
    """Operands and result inside wider buffers; nothing outside is touched;
    another stream; a caller's workspace."""
    a, b = _operands(cuda_lib, "nt", 70, 200, 300, 50, lambda s, seed: _rand(s, torch.float32, seed))
    want = cuda_lib.kda_fp8_matmul(a, b, "nt", out_dtype=torch.float32)
    wide = torch.full((70, 512), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    wide.view(torch.uint8)[:, :300] = a.data.view(torch.uint8)
    aw = cuda_lib.Fp8Matrix(wide[:, :300], a.scales, "row")
    for dtype in (torch.float32, torch.bfloat16):
        buf = torch.full((72, 333), 7.0, dtype=dtype, device="cuda")
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        cuda_lib.kda_fp8_matmul(aw, b, "nt", out=buf[1:71, 5:205], workspace=ws, stream=side)
        side.synchronize()
        assert torch.equal(buf[1:71, 5:205], want.to(dtype))
        buf[1:71, 5:205] = 7.0
        assert torch.all(buf == 7.0)
        assert cuda_lib.kda_get_device_status(ws) == cuda_lib.KDA_OK


def test_matmul_nan_stays_in_its_row_and_column(cuda_lib):
    x, w = _rand((40, 256), torch.float32, 60), _rand((130, 256), torch.float32, 61)
    x[3, 100], w[129, 7] = float("nan"), float("inf")
    a, = cuda_lib.kda_fp8_quantize(x)
    b, = cuda_lib.kda_fp8_quantize(w, kinds="tile")
    got = cuda_lib.kda_fp8_matmul(a, b)
    bad = torch.isnan(got)
    want = torch.zeros_like(bad)
    want[3], want[:, 129] = True, True
    assert torch.equal(bad, want)


def test_matmul_empty(cuda_lib):
    make = lambda s, seed: _rand(s, torch.float32, seed) if s[0] else torch.zeros(s, device="cuda")  # noqa: E731
    a, b = _operands(cuda_lib, "nt", 0, 100, 64, 70, make)
    assert cuda_lib.kda_fp8_matmul(a, b).shape == (0, 100)
    a, = cuda_lib.kda_fp8_quantize(torch.zeros(0, 48, device="cuda"), kinds="col")
    b, = cuda_lib.kda_fp8_quantize(torch.zeros(0, 80, device="cuda"), kinds="col")
    out = torch.full((48, 80), 7.0, device="cuda")
    cuda_lib.kda_fp8_matmul(a, b, "tn", out=out)
    assert float(out.abs().max()) == 0


def test_matmul_in_a_graph(cuda_lib):
    a, b = _operands(cuda_lib, "nt", 3, 512, 1024, 80, lambda s, seed: _rand(s, torch.float32, seed))
    want = cuda_lib.kda_fp8_matmul(a, b)
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cuda_lib.kda_fp8_matmul(a, b, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("m,n,k", [(3, 512, 2048), (2500, 2600, 272)])
def test_matmul_wait_that_runs_out_is_reported(cuda_lib, m, n, k):
    """Both kernels (k split over a cluster; pairs of CTAs) end in bounded
    time, report it, and the next call is right."""
    a, b = _operands(cuda_lib, "nt", m, n, k, 90, lambda s, seed: _rand(s, torch.float32, seed))
    want = cuda_lib.kda_fp8_matmul(a, b)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    cuda_lib.kda_fp8_matmul(a, b, workspace=ws, extra_flags=cuda_lib.KDA_TEST_WAIT_TIMEOUT)
    assert cuda_lib.kda_get_device_status(ws) == cuda_lib.KDA_ERR_DEVICE_TIMEOUT
    assert cuda_lib.kda_get_device_status(ws) == cuda_lib.KDA_OK
    assert torch.equal(cuda_lib.kda_fp8_matmul(a, b, workspace=ws), want)
    assert cuda_lib.kda_get_device_status(ws) == cuda_lib.KDA_OK


def test_offsets_beyond_32_bits(cuda_lib):
    """Rows whose elements and bytes lie past 2^31 and 2^32: the last ones
    equal the same rows worked alone."""
    rows, cols = 1_050_000, 2056   # 2.2e9 elements
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-300:] = _rand((300, cols), torch.bfloat16, 100)
    x[:300] = x[-300:]
    got = cuda_lib.kda_rms_norm(x, None, fp8=True)
    alone = cuda_lib.kda_rms_norm(x[-300:].clone(), None, fp8=True)
    for part in (got.out[-300:], got.out[:300]):
        assert torch.equal(part, alone.out)
    assert torch.equal(got.fp8.data[-300:].view(torch.uint8), alone.fp8.data.view(torch.uint8))
    assert torch.equal(got.fp8.scales[:, -300:].view(torch.uint8), alone.fp8.scales.view(torch.uint8))
    dx, _ = cuda_lib.kda_rms_norm_bwd(got.out, x)
    dx_alone, _ = cuda_lib.kda_rms_norm_bwd(alone.out, x[-300:].clone())
    assert torch.equal(dx[-300:], dx_alone)
    del dx, got
    row, = cuda_lib.kda_fp8_quantize(x)
    row_alone, = cuda_lib.kda_fp8_quantize(x[-300:].clone())
    assert torch.equal(row.data[-300:].view(torch.uint8), row_alone.data.view(torch.uint8))
    w, = cuda_lib.kda_fp8_quantize(_rand((2304, cols), torch.float32, 101), kinds="tile")
    y = cuda_lib.kda_fp8_matmul(row, w)   # 2.4e9 outputs
    y_alone = cuda_lib.kda_fp8_matmul(row_alone, w, out_dtype=torch.float32)
    # the two kernels may sum in another order
    d = (y[-300:].float() - y_alone).abs().max()
    assert float(d) <= float(y_alone.abs().max()) * 2 * U16
    assert torch.equal(y[-300:], y[:300])


def test_calls_in_a_row_keep_their_order(cuda_lib):
    """Each kernel is set up while the one before it ends: a chain of calls,
    each on the last one's results and some in place, gives bit for bit what
    it gives with a synchronisation after every call; torch's own kernels in
    between."""
    w, = cuda_lib.kda_fp8_quantize(_rand((1024, 1024), torch.float32, 110) / 32, kinds="tile")
    x0, r0 = _rand((700, 1024), torch.bfloat16, 111), _rand((700, 1024), torch.bfloat16, 112)

    def chain(wait):
        x, r, total = x0.clone(), r0.clone(), torch.zeros(1024, 1024, device="cuda")
        for i in range(12):
            n = cuda_lib.kda_rms_norm(x, None, r, fp8=True, residual_out=r)
            wait()
            x = cuda_lib.kda_fp8_matmul(n.fp8, w)
            wait()
            row, col = cuda_lib.kda_fp8_quantize(x, ("row", "col"))
            wait()
            g = cuda_lib.kda_fp8_matmul(row, w, "nn")
            wait()
            g, dw = cuda_lib.kda_rms_norm_bwd(g, r, None, x, dx=g)
            wait()
            n_col, = cuda_lib.kda_fp8_quantize(n.out, "col")
            total += cuda_lib.kda_fp8_matmul(col, n_col, "tn", out_dtype=torch.float32)
            wait()
            x = (x.float() * 0.5 + g.float() + dw * 1e-3).bfloat16()
        return x, r, total

    want = chain(torch.cuda.synchronize)
    for _ in range(3):
        for a, b in zip(chain(lambda: None), want):
            assert torch.equal(a, b)
