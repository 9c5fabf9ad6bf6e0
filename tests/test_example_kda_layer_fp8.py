"""The example layer (examples/kda_layer_fp8.py) against the same layer in 64
bits without 8-bit rounding: KDA from the oracle, everything else in numpy."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
H, B, T = 2, 1, 150
# e4m3 rounds a value by at most 2^-4 of it, 2^-4 / 3^(1/2) / 2^(1/2) in the mean square over a
# binade (2.6%); a product of two such operands is 3.6% off, and the output passes through two of
# them: 5.1%.  KDA's quotients and gates (q and k normalised, the gate an exponent) add the error
# of four more inputs at most linearly.
TOL_Y = 0.15
# a gradient passes through three products more
TOL_GRAD = 0.3


def _example():
    spec = importlib.util.spec_from_file_location("kda_layer_fp8", os.path.join(ROOT, "examples", "kda_layer_fp8.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _rel(x, y):
    return float(np.linalg.norm(_np(x).reshape(y.shape) - y) / np.linalg.norm(y))


@pytest.fixture(scope="module")
def layer(cuda_lib):
    ex = _example()
    return ex.KdaLayerFp8(H, ex.random_weights(H, torch.device("cuda"), seed=1))


def _inputs(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(B, T, H * 128, device="cuda", generator=g).bfloat16() for _ in range(4)]


def _reference(layer, x, r, s0):
    """The layer in 64 bits, and what its backward needs."""
    w = {n: _np(t) for n, t in layer.w.items()}
    h = _np((x.float() + r.float()).bfloat16()).reshape(T, -1)
    rstd = 1 / np.sqrt((h * h).mean(1, keepdims=True) + 1e-6)
    n = h * rstd * w["norm"]
    p = {k: n @ w[k].T for k in layer.IN}
    prob = oracle.Problem(*(p[k].reshape(T, H, 128) for k in ("q", "k", "v", "gate")), p["beta"].reshape(T, H),
                          cu_seqlens=[0, T], scale=128 ** -0.5, eps=1e-6, a_log=w["a_log"], dt_bias=w["dt_bias"],
                          l2norm=True, beta_sigmoid=True, gate_in_kernel=True)
    o, s = oracle.chunk_fwd(prob, s0)
    return w, h, rstd, n, prob, o.reshape(T, -1), s


def test_prefill_and_backward(layer, cuda_lib):
    x, r, dy, ds = _inputs(2)
    s0 = 0.1 * torch.randn(B, H, 128, 128, device="cuda")
    y, stream, state, kept = layer.prefill(x, r, s0, keep=True)
    w, h, rstd, n, prob, o, s = _reference(layer, x, r, _np(s0))
    assert torch.equal(stream, (x.float() + r.float()).bfloat16())
    assert _rel(y, o @ w["out"].T) <= TOL_Y
    assert _rel(state, s) <= TOL_Y
    short = layer.prefill(x, r, s0)
    assert torch.equal(short[0], y) and torch.equal(short[2], state)

    dx, grads = layer.backward(kept, dy, ds)
    DY, DS = _np(dy).reshape(T, -1), _np(ds).reshape(T, -1)
    g = oracle.chunk_bwd(prob, _np(s0), (DY @ w["out"]).reshape(T, H, 128), None)
    flat = dict(q=g["dq"], k=g["dk"], v=g["dv"], gate=g["dg"], beta=g["dbeta"])
    flat = {k: np.asarray(v).reshape(T, -1) for k, v in flat.items()}
    want = {k: v.T @ n for k, v in flat.items()}
    want["out"] = DY.T @ o
    dn = sum(flat[k] @ w[k] for k in layer.IN)
    want["norm"] = (dn * h * rstd).sum(0)
    gw, nn = dn * w["norm"], h * rstd
    want_x = rstd * (gw - nn * (gw * nn).mean(1, keepdims=True)) + DS
    assert _rel(dx, want_x) <= TOL_GRAD
    for k, v in want.items():
        assert _rel(grads[k], v) <= TOL_GRAD, k
    assert cuda_lib.kda_fp8_matmul_status() == cuda_lib.KDA_OK


def test_decode_continues_a_prefill(layer):
    """Rows are quantised one by one, so a token's projections do not depend on
    its neighbours: decode differs from prefill only in KDA's own two forms."""
    x, r, _, _ = _inputs(3)
    y, stream, state = layer.prefill(x, r)
    half = T // 2
    _, _, s = layer.prefill(x[:, :half].contiguous(), r[:, :half].contiguous())
    pool = torch.randn(5, H, 128, 128, device="cuda")
    rows = torch.tensor([3], dtype=torch.int32, device="cuda")
    pool[3] = s[0]
    out = []
    for t in range(half, T):
        y_t, stream_t = layer.decode(x[:, t].contiguous(), r[:, t].contiguous(), pool, rows)
        assert torch.equal(stream_t, stream[:, t])
        out.append(y_t)
    # o of the two forms agrees to bf16's 2e-2 (the library's tolerance); its 8-bit rounding adds
    # a step of e4m3 where the two fall on different sides
    assert _rel(torch.stack(out, 1), _np(y[:, half:])) <= 4e-2
    assert _rel(pool[3], _np(state[0])) <= 2e-2
