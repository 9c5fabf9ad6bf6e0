"""The 8-bit projection path around a KDA layer, as cases to measure: the RMS norm that adds the
residual and leaves 8-bit values with scales (and its backward), the quantiser, and the matrix product
of 8-bit operands with a scale for each block of 128.

8-bit values are e4m3; scales are powers of two, one byte (exponent + 127) each.  Three kinds of
scaled matrix [R, C]:
  row   one scale for 128 consecutive columns of a row, stored [ceil(CB / 4), R, 4] with CB = ceil(C / 128)
  col   one scale for 128 consecutive rows of a column, stored [ceil(RB / 4), C, 4] with RB = ceil(R / 128)
  tile  one scale for a 128 x 128 block, stored [RB, CB]
Entries past the last block are 1.0.  The values are [R, C] with a row pitch that is a multiple of 16.

Cases are dicts: "op" is norm, norm_bwd, quantize or matmul; the other keys are its sizes and options.
"""
import math

import torch
import torch.nn.functional as F

own = False

EPS = 1e-6
# a drawn case costs no more than the largest listed ones: elements of a norm or a quantiser, products of a matmul
MOST_ELEMS = 32768 * 4096
MOST_MACS = 32768 * 4096 * 4096


def listed():
    return [
        # one token of one sequence in decode, width 32 heads x 128: latency of a single row
        dict(name="norm_token", op="norm", rows=1, cols=4096, dtype="bf16", residual=True, out="fp8"),
        # prefill of 2 x 4096 tokens, width 16 heads x 128: the layer's entry in ordinary serving
        dict(name="norm_prefill", op="norm", rows=8192, cols=2048, dtype="bf16", residual=True, out="fp8"),
        # packed sequences of odd total length, a width that is no multiple of anything, fp32 activations, no residual
        dict(name="norm_ragged_f32", op="norm", rows=4099, cols=1111, dtype="f32", residual=False, out="same"),
        # the training batch of 4 x 8192 tokens, width 32 heads x 128
        dict(name="norm_train", op="norm", rows=32768, cols=4096, dtype="bf16", residual=True, out="fp8"),
        # its backward pass: the gradients of the input (residual's gradient added) and of the weight
        dict(name="norm_train_bwd", op="norm_bwd", rows=32768, cols=4096, dtype="bf16", residual=True),
        # an activation of the training batch for the forward product (row) and the weight gradient (col), at once
        dict(name="quantize_train", op="quantize", rows=32768, cols=4096, dtype="bf16", kinds="row,col"),
        # a master weight after an optimiser step, with an output width of 32 heads x 128 + 100
        dict(name="quantize_weight", op="quantize", rows=4196, cols=4096, dtype="f32", kinds="tile"),
        # one token through a projection of 32 heads x 128: the weight's bytes
        dict(name="matmul_token", op="matmul", form="nt", m=1, n=4096, k=4096, out="bf16"),
        # a packed prefill of few tokens, odd sizes everywhere, a last block of 16 columns
        dict(name="matmul_ragged", op="matmul", form="nt", m=777, n=1111, k=2064, out="bf16"),
        # the training batch through a projection: the forward product
        dict(name="matmul_train", op="matmul", form="nt", m=32768, n=4096, k=4096, out="bf16"),
        # the input's gradient, prefill-sized batch
        dict(name="matmul_dgrad", op="matmul", form="nn", m=8192, n=2048, k=4096, out="bf16"),
        # the weight's gradient over 8200 packed tokens (a last block of 8), kept in fp32
        dict(name="matmul_wgrad", op="matmul", form="tn", m=4096, n=2048, k=8200, out="f32"),
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng):
    """A width between 64 and 8200: an odd number of whole blocks, a multiple of 8 with part of a block at the end, or odd."""
    w = _log_uniform(rng, 64, 8192)
    return rng.choice([w // 256 * 256 + 128, w // 256 * 256 + 128, w // 16 * 16 + 8, w | 1])


def _rows(rng, most):
    """An odd number of rows up to 32767 and `most`: packed sequences seldom add up to a round number."""
    return (min(_log_uniform(rng, 1, 32768), max(1, most)) - 1) | 1


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "quantize", "matmul", "matmul", "matmul"])
    if op == "matmul":
        form = rng.choice(["nt", "nt", "nn", "tn"])
        wide, inner = _width(rng), _width(rng)
        rows = _rows(rng, MOST_MACS // (wide * inner) - 1)
        if form == "tn":  # rows are the tokens that the product sums over
            return dict(op=op, form=form, m=wide, n=inner, k=rows, out="f32")
        return dict(op=op, form=form, m=rows, n=wide, k=inner, out="bf16")
    cols = _width(rng)
    rows = _rows(rng, MOST_ELEMS // cols - 1)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, residual=rng.random() < 0.7, out=rng.choice(["fp8", "fp8", "same"]))
    if op == "norm_bwd":
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, residual=rng.random() < 0.7)
    return dict(op=op, rows=rows, cols=cols, dtype=dtype, kinds=rng.choice(["row", "row,col", "col", "tile"]))


# ---------------------------------------------------------------- plain form

def _dtype(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _blocks(n):
    return -(-n // 128)


def _pad_blocks(x):
    """[R, C] with zeros up to whole blocks, as [RB, 128, CB, 128]."""
    r, c = x.shape
    x = F.pad(x, (0, _blocks(c) * 128 - c, 0, _blocks(r) * 128 - r))
    return x.view(_blocks(r), 128, _blocks(c), 128)


def _block_exponent(amax):
    """The smallest e >= -127 with amax <= 448 * 2^e (448 is the largest e4m3 value); 0 for a block of zeros."""
    m, ex = torch.frexp(amax)
    e = ex - 9 + (m > 0.875).to(ex.dtype)
    return torch.where(amax > 0, e.clamp(min=-127), torch.zeros_like(e))


def _pack(e, kind):
    """Exponents [RB or R, CB or C] as the stored scales."""
    b = (e + 127).to(torch.uint8)
    if kind != "tile":
        b = b if kind == "row" else b.t()
        n = -(-b.shape[1] // 4) * 4
        b = F.pad(b, (0, n - b.shape[1]), value=127).view(b.shape[0], n // 4, 4).permute(1, 0, 2).contiguous()
    return b.view(torch.float8_e8m0fnu)


def _scaled(x, kind):
    """fp32 [R, C] -> (values in the range of e4m3 before rounding, stored scales)."""
    r, c = x.shape
    p = _pad_blocks(x)
    dims = {"row": (3,), "col": (1,), "tile": (1, 3)}[kind]
    amax = torch.where(torch.isfinite(p), p.abs(), torch.zeros_like(p)).amax(dims, keepdim=True)
    e = _block_exponent(amax)
    v = (p * torch.exp2(-e.float())).view(p.shape[0] * 128, -1)[:r, :c]
    e = {"row": lambda: e.reshape(-1, e.shape[2])[:r], "col": lambda: e.reshape(e.shape[0], -1)[:, :c], "tile": lambda: e[:, 0, :, 0]}[kind]()
    return v, _pack(e, kind)


def _quantize(x, kind):
    v, scales = _scaled(x, kind)
    r, c = v.shape
    data = torch.zeros(r, -(-c // 16) * 16, dtype=torch.float8_e4m3fn, device=x.device)
    data[:, :c] = v.to(torch.float8_e4m3fn)
    return data[:, :c], scales


def _dequantize(data, scales, kind):
    r, c = data.shape
    e = scales.view(torch.uint8).float() - 127
    if kind != "tile":
        e = e.permute(1, 0, 2).flatten(1)
        e = e[:, :_blocks(c)] if kind == "row" else e[:, :_blocks(r)].t()
    s = torch.exp2(e)
    if kind != "row":
        s = s.repeat_interleave(128, 0)[:r]
    if kind != "col":
        s = s.repeat_interleave(128, 1)[:, :c]
    return data.float() * s


_KINDS = {"nt": ("row", "tile"), "nn": ("row", "tile"), "tn": ("col", "col")}


def _shapes(case):
    m, n, k = case["m"], case["n"], case["k"]
    return {"nt": ((m, k), (n, k)), "nn": ((m, k), (k, n)), "tn": ((k, m), (k, n))}[case["form"]]


# ---------------------------------------------------------------- inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) % (1 << 62))


def _activations(g, r, c, dtype):
    """Rows of different size and a few channels far above the others, as a residual stream has them."""
    x = torch.randn(r, c, device="cuda", generator=g)
    x *= torch.exp(0.5 * torch.randn(r, 1, device="cuda", generator=g))
    x *= 1 + 15 * (torch.rand(1, c, device="cuda", generator=g) < 0.005)
    return x.to(dtype)


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "matmul":
        (ra, ca), (rb, cb) = _shapes(case)
        ka, kb = _KINDS[case["form"]]
        a = _quantize(_activations(g, ra, ca, torch.float32), ka)
        b = torch.randn(rb, cb, device="cuda", generator=g) * 0.02 if kb == "tile" else _activations(g, rb, cb, torch.float32)
        return dict(case=case, a=a, b=_quantize(b, kb))
    dtype = _dtype(case["dtype"])
    s = dict(case=case, x=_activations(g, case["rows"], case["cols"], dtype))
    if case["op"] == "quantize":
        if case["kinds"] == "tile":  # a weight
            s["x"] = (torch.randn(case["rows"], case["cols"], device="cuda", generator=g) * 0.02).to(dtype)
        return s
    s["weight"] = 1 + 0.1 * torch.randn(case["cols"], device="cuda", generator=g)
    s["residual"] = s["d_residual"] = None
    if case["op"] == "norm":
        if case["residual"]:
            s["residual"] = _activations(g, case["rows"], case["cols"], dtype)
        return s
    s["d_out"] = torch.randn(case["rows"], case["cols"], device="cuda", generator=g).to(dtype)
    if case["residual"]:
        s["d_residual"] = torch.randn(case["rows"], case["cols"], device="cuda", generator=g).to(dtype)
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import chunked_kimi_delta_gb300 as kda
    case = s["case"]
    if case["op"] == "norm":
        out = kda.kda_rms_norm(s["x"], s["weight"], s["residual"], eps=EPS, fp8=case["out"] == "fp8", out=None if case["out"] == "same" else False)
        y = [out.out] if case["out"] == "same" else [out.fp8.data, out.fp8.scales]
        return y + ([out.residual_out] if case["residual"] else [])
    if case["op"] == "norm_bwd":
        return list(kda.kda_rms_norm_bwd(s["d_out"], s["x"], s["weight"], s["d_residual"], eps=EPS))
    if case["op"] == "quantize":
        parts = kda.kda_fp8_quantize(s["x"], kinds=case["kinds"].split(","))
        return [t for p in parts for t in (p.data, p.scales)]
    ka, kb = _KINDS[case["form"]]
    return kda.kda_fp8_matmul(kda.Fp8Matrix(*s["a"], ka), kda.Fp8Matrix(*s["b"], kb), form=case["form"], out_dtype=_dtype(case["out"]))


def _run_plain(s):
    case = s["case"]
    if case["op"] == "norm":
        h = s["x"].float() if s["residual"] is None else s["x"].float() + s["residual"].float()
        h = h.to(s["x"].dtype)  # the sum as it is kept for the next layer is what is normalised
        f = h.float()
        y = f * torch.rsqrt((f * f).mean(1, keepdim=True) + EPS) * s["weight"]
        y = [y.to(h.dtype)] if case["out"] == "same" else list(_quantize(y, "row"))
        return y + ([h] if case["residual"] else [])
    if case["op"] == "norm_bwd":
        f, gy = s["x"].float(), s["d_out"].float()
        rstd = torch.rsqrt((f * f).mean(1, keepdim=True) + EPS)
        n = f * rstd
        gn = gy * s["weight"]
        dx = rstd * (gn - n * (gn * n).mean(1, keepdim=True))
        if s["d_residual"] is not None:
            dx = dx + s["d_residual"].float()
        return [dx.to(s["x"].dtype), (gy * n).sum(0)]
    if case["op"] == "quantize":
        x = s["x"].float()
        return [t for kind in case["kinds"].split(",") for t in _quantize(x, kind)]
    ka, kb = _KINDS[case["form"]]
    a, b = _dequantize(*s["a"], ka), _dequantize(*s["b"], kb)
    a = a.t() if case["form"] == "tn" else a
    b = b.t() if case["form"] == "nt" else b
    return torch.matmul(a, b).to(_dtype(case["out"]))


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    if case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        scales = {"row": lambda r, c: r * _blocks(c), "col": lambda r, c: _blocks(r) * c, "tile": lambda r, c: _blocks(r) * _blocks(c)}
        operands = sum(r * c + scales[kind](r, c) for (r, c), kind in zip(_shapes(case), _KINDS[case["form"]]))
        return dict(bytes=operands + m * n * (2 if case["out"] == "bf16" else 4), flops=2.0 * m * n * k)
    r, c, e = case["rows"], case["cols"], 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        out = r * c * e if case["out"] == "same" else r * c + r * _blocks(c)
        return dict(bytes=r * c * e * (3 if case["residual"] else 1) + 4 * c + out, flops=5.0 * r * c)
    if case["op"] == "norm_bwd":
        return dict(bytes=r * c * e * (4 if case["residual"] else 3) + 8 * c, flops=12.0 * r * c)
    per = {"row": r * _blocks(c), "col": _blocks(r) * c, "tile": _blocks(r) * _blocks(c)}
    kinds = case["kinds"].split(",")
    return dict(bytes=r * c * e + sum(r * c + per[kind] for kind in kinds), flops=3.0 * r * c * len(kinds))


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_e4m3(v):
    """v in fp64, |v| <= 448, rounded to the nearest e4m3 value (ties to even; 2^-9 is the smallest step)."""
    step = torch.ldexp(torch.ones_like(v), (torch.frexp(v)[1] - 4).clamp(min=-9))
    return torch.round(v / step) * step


def _exact_quantize(x, kind):
    """fp64 [R, C] -> [e4m3 values, stored scales], from the definition: 2^e is the smallest power of two with max|x| <= 448 * 2^e."""
    r, c = x.shape
    br, bc = {"row": (1, 128), "col": (128, 1), "tile": (128, 128)}[kind]
    nr, nc = -(-r // br), -(-c // bc)
    full = torch.zeros(nr * br, nc * bc, dtype=torch.float64, device=x.device)
    full[:r, :c] = x
    top = full.abs().view(nr, br, nc, bc).amax((1, 3))
    e = torch.ceil(torch.log2(torch.where(top > 0, top, torch.full_like(top, 448.0)) / 448))
    e = torch.where(top > 448 * torch.exp2(e), e + 1, e)
    e = torch.where(top <= 448 * torch.exp2(e - 1), e - 1, e)
    s = torch.exp2(torch.where(top > 0, e, torch.zeros_like(e)).clamp(min=-127.0))
    values = _exact_e4m3(full / s.repeat_interleave(br, 0).repeat_interleave(bc, 1))[:r, :c]
    if kind != "tile":
        s = s if kind == "row" else s.t()
        words = torch.ones(s.shape[0], -(-s.shape[1] // 4) * 4, dtype=torch.float64, device=x.device)
        words[:, :s.shape[1]] = s
        s = words.view(s.shape[0], -1, 4).permute(1, 0, 2).contiguous()
    return [values, s]


def _exact_values(data, scales, kind):
    r, c = data.shape
    s = torch.exp2(scales.view(torch.uint8).double() - 127)
    i = torch.arange(r, device=data.device)[:, None].expand(r, c)
    j = torch.arange(c, device=data.device)[None, :].expand(r, c)
    if kind == "row":
        s = s[j // 512, i, j // 128 % 4]
    elif kind == "col":
        s = s[i // 512, j, i // 128 % 4]
    else:
        s = s[i // 128, j // 128]
    return data.double() * s


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "matmul":
        a, b = (_exact_values(*s[key], kind) for key, kind in zip("ab", _KINDS[case["form"]]))
        if case["form"] == "nt":
            return a @ b.t()
        return a @ b if case["form"] == "nn" else a.t() @ b
    x = s["x"].double()
    if case["op"] == "quantize":
        return [t for kind in case["kinds"].split(",") for t in _exact_quantize(x, kind)]
    w, d = s["weight"].double(), case["cols"]
    if case["op"] == "norm":
        total = x if s["residual"] is None else x + s["residual"].double()
        h = total.to(s["x"].dtype).double()
        y = h / torch.sqrt(h.square().sum(1, keepdim=True) / d + EPS) * w
        return ([y] if case["out"] == "same" else _exact_quantize(y, "row")) + ([total] if case["residual"] else [])
    g = s["d_out"].double()
    scale = 1 / torch.sqrt(x.square().sum(1, keepdim=True) / d + EPS)
    dx = scale * g * w - x * scale ** 3 * (g * w * x).sum(1, keepdim=True) / d
    if s["d_residual"] is not None:
        dx = dx + s["d_residual"].double()
    return [dx, (g * x * scale).sum(0)]
