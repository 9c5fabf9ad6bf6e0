"""A KDA layer with 8-bit projections, put together from the library's calls:
prefill, one-token decode on a state pool, and a training step's gradients.

    h   = x + residual                      kda_rms_norm (adds, normalises, quantises)
    q, k, v, gate, beta = norm(h) W^T       kda_fp8_matmul "nt", 8-bit in, bf16 / fp32 out
    o   = KDA(q, k, v, gate, beta)          kda_chunk_fwd, or kda_recurrent_step
    y   = o W_out^T                         kda_fp8_quantize, kda_fp8_matmul "nt"

Backward: gradients of y and of the residual stream in, of x (and residual),
the weights and the gate's parameters out; every product in 8 bits ("nn" for
the inputs, "tn" over the tokens for the weights), each gradient quantised
once for both of its products.

Run it (GB300): python examples/kda_layer_fp8.py
"""
from __future__ import annotations

import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import chunked_kimi_delta_gb300 as kda

EPS = 1e-6
_GATES = dict(gate_in_kernel=True, beta_sigmoid=True)


class KdaLayerFp8:
    """heads x 128 channels wide.  ``weights`` holds fp32 master weights:
    norm [D], q, k, v, gate, out [D, D], beta [heads, D], a_log [heads],
    dt_bias [heads, 128]."""

    IN = ("q", "k", "v", "gate", "beta")

    def __init__(self, heads: int, weights: dict):
        self.heads, self.width, self.w = heads, heads * 128, weights
        self.quantize_weights()

    def quantize_weights(self):
        """After every change of the master weights."""
        self.w8 = {n: kda.kda_fp8_quantize(self.w[n], "tile")[0] for n in (*self.IN, "out")}

    def _project(self, n8, lead):
        """The five projections of the normalised input, in KDA's layouts."""
        out = {n: kda.kda_fp8_matmul(n8, self.w8[n], out_dtype=torch.float32 if n in ("gate", "beta") else torch.bfloat16)
               for n in self.IN}
        return {n: t.view(*lead, self.heads) if n == "beta" else t.view(*lead, self.heads, 128) for n, t in out.items()}

    def _gate_params(self):
        return dict(a_log=self.w["a_log"], dt_bias=self.w["dt_bias"], **_GATES)

    def prefill(self, x, residual, initial_state=None, keep=False):
        """x, residual [B, T, D] bf16.  Returns (y, residual stream, final
        state [B, heads, 128, 128]) and, with ``keep``, what backward needs."""
        B, T, D = x.shape
        n = kda.kda_rms_norm(x, self.w["norm"], residual, eps=EPS, fp8=True, out=None if keep else False)
        p = self._project(n.fp8, (B, T))
        o, state = kda.kda_chunk_fwd(p["q"], p["k"], p["v"], p["gate"], p["beta"], initial_state=initial_state,
                                     **self._gate_params())
        o = o.view(B * T, D)
        o8, = kda.kda_fp8_quantize(o)
        y = kda.kda_fp8_matmul(o8, self.w8["out"]).view(B, T, D)
        if not keep:
            return y, n.residual_out, state
        return y, n.residual_out, state, dict(n=n.out.view(B * T, D), h=n.residual_out, p=p, o=o, initial_state=initial_state)

    def decode(self, x, residual, pool, rows):
        """One token for each sequence: x, residual [N, D]; the states are the
        rows ``rows`` [N] of ``pool`` [., heads, 128, 128], updated in place."""
        N, D = x.shape
        n = kda.kda_rms_norm(x, self.w["norm"], residual, eps=EPS, fp8=True, out=False)
        p = self._project(n.fp8, (N, 1))
        o = kda.kda_recurrent_step(p["q"], p["k"], p["v"], p["gate"], p["beta"], pool, rows, **self._gate_params())
        o8, = kda.kda_fp8_quantize(o.view(N, D))
        return kda.kda_fp8_matmul(o8, self.w8["out"]), n.residual_out

    def backward(self, kept, d_y, d_stream):
        """d_y, d_stream [B, T, D]: gradients of y and of the residual stream.
        Returns (gradient of x and of residual, dict of weight gradients)."""
        D = self.width
        tn = dict(form="tn", out_dtype=torch.float32)
        d_row, d_col = kda.kda_fp8_quantize(d_y.view(-1, D), ("row", "col"))
        o_col, n_col = kda.kda_fp8_quantize(kept["o"], "col")[0], kda.kda_fp8_quantize(kept["n"], "col")[0]
        grads = {"out": kda.kda_fp8_matmul(d_col, o_col, **tn)}
        p = kept["p"]
        d_o = kda.kda_fp8_matmul(d_row, self.w8["out"], "nn").view(p["v"].shape)
        g = kda.kda_chunk_bwd(p["q"], p["k"], p["v"], p["gate"], p["beta"], d_o, initial_state=kept["initial_state"],
                              **self._gate_params())
        grads["a_log"], grads["dt_bias"] = g["da_log"], g["ddt_bias"]
        d_n = None
        for name, key in zip(self.IN, ("dq", "dk", "dv", "dg", "dbeta")):
            d_row, d_col = kda.kda_fp8_quantize(g[key].view(kept["n"].shape[0], -1), ("row", "col"))
            grads[name] = kda.kda_fp8_matmul(d_col, n_col, **tn)
            part = kda.kda_fp8_matmul(d_row, self.w8[name], "nn", out_dtype=torch.float32)
            d_n = part if d_n is None else d_n.add_(part)
        d_n = d_n.to(torch.bfloat16).view(kept["h"].shape)
        d_x, grads["norm"] = kda.kda_rms_norm_bwd(d_n, kept["h"], self.w["norm"], d_stream, eps=EPS)
        return d_x, grads


def random_weights(heads, device, seed=0):
    g = torch.Generator(device=device).manual_seed(seed)
    D = heads * 128
    normal = lambda *s: torch.randn(*s, device=device, generator=g)  # noqa: E731
    w = {n: normal(D, D) * D ** -0.5 for n in ("q", "k", "v", "gate", "out")}
    w["beta"] = normal(heads, D) * D ** -0.5
    w["norm"] = 1 + 0.1 * normal(D)
    w["a_log"] = -4 * torch.rand(heads, device=device, generator=g)
    w["dt_bias"] = 0.1 * normal(heads, 128)
    return w


def main():
    heads, B, T = 16, 2, 4096
    dev = torch.device("cuda")
    layer = KdaLayerFp8(heads, random_weights(heads, dev))
    x = torch.randn(B, T, layer.width, device=dev).bfloat16()
    r = torch.randn(B, T, layer.width, device=dev).bfloat16()
    d = torch.randn(B, T, layer.width, device=dev).bfloat16()
    pool, rows = torch.zeros(B, heads, 128, 128, device=dev), torch.arange(B, dtype=torch.int32, device=dev)

    def timed(what, f, n=10):
        for _ in range(3):
            f()
        e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        e[0].record()
        for _ in range(n):
            f()
        e[1].record()
        torch.cuda.synchronize()
        print(f"{what}: {e[0].elapsed_time(e[1]) / n * 1e3:.0f} us")

    timed(f"prefill of {B} x {T} tokens, {heads} heads", lambda: layer.prefill(x, r))
    _, _, state, kept = layer.prefill(x, r, keep=True)
    pool.copy_(state)
    timed("forward kept for backward", lambda: layer.prefill(x, r, keep=True))
    timed("backward", lambda: layer.backward(kept, d, d))
    timed(f"decode, {B} sequences", lambda: layer.decode(x[:, -1].contiguous(), r[:, -1].contiguous(), pool, rows))
    assert kda.kda_fp8_matmul_status() == kda.KDA_OK


if __name__ == "__main__":
    main()
