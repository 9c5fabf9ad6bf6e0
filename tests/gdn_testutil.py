"""The gated delta rule with one gate per head: seeded problems, the library's
calls on them and the 64-bit oracle (the per-channel recurrence with the gate
repeated over the channels; gradients of a head's gate are the sums over them).

Tolerances, relative to the 2-norm of the whole result:
  bf16 results  one rounding, at most half a step of 2^-8 relative, plus operands rounded to 11 bits
                (2^-12 each, two products in a row): below 2^-8 + 4 * 2^-12 = 4.9e-3
  fp32 results  operands keep 22 bits (two a product, at most 2^-22 each); a tensor-core step drops
                less than 2^-23 of its running sum and a sum takes at most 24 steps; four products in a
                row (k S, A Y, W^T k and the next chunk's k S) decide a chunk's state:
                4 * (2 * 2^-22 + 24 * 2^-23) = 1.4e-5 at worst, all errors of one sign; errors are not,
                so a half of that is asked for: 7e-6
"""
from __future__ import annotations

import numpy as np
import torch

import oracle

TOL = {torch.bfloat16: 2.0 ** -8 + 4 * 2.0 ** -12, torch.float32: 7e-6}
EPS = float(np.float32(1e-6))


def problem(lens, *, hk=2, h=4, dk=128, dv=128, dtype=torch.bfloat16, packed=None, gate="slow", initial=True, seed=0,
            raw=False):
    """Inputs on the CPU; raw: beta, log-decay and keys of modest size are given as they are used."""
    gen = torch.Generator().manual_seed(seed)

    def randn(*s):
        return torch.randn(*s, generator=gen)
    packed = len(set(lens)) > 1 if packed is None else packed
    lead = (sum(lens),) if packed else (len(lens), lens[0])
    p = dict(q=randn(*lead, hk, dk).to(dtype), k=randn(*lead, hk, dk).to(dtype), v=randn(*lead, h, dv).to(dtype),
             g=randn(*lead, h), beta=randn(*lead, h))
    cu = np.concatenate([[0], np.cumsum(lens)])
    kw = dict(scale=float(np.float32(dk ** -0.5)), eps=EPS, initial_state=0.1 * randn(len(lens), h, dk, dv) if initial else None,
              cu_seqlens=torch.tensor(cu, dtype=torch.int32) if packed else None)
    lo, hi = {"slow": (-4.0, 0.0), "strong": (1.0, 3.0)}[gate]
    a_log, dt_bias = lo + (hi - lo) * torch.rand(h, generator=gen), 0.1 * randn(h)
    d_out, d_final = randn(*lead, h, dv).to(dtype), 0.1 * randn(len(lens), h, dk, dv)
    if raw:
        p["g"], p["beta"] = -p["g"].abs() * (0.1 if gate == "slow" else 3.0), torch.sigmoid(p["beta"])
        p["k"] = (p["k"].float() * 0.07).to(dtype)
        kw.update(l2norm_qk=False)
    else:
        kw.update(a_log=a_log, dt_bias=dt_bias, beta_sigmoid=True, gate_in_kernel=True)
    return dict(p, kw=kw, cu=cu, d_out=d_out, d_final=d_final)


def oracle_of(p):
    """oracle.Problem with the gate and the key heads repeated."""
    h, hk, dk = p["v"].shape[-2], p["q"].shape[-2], p["q"].shape[-1]
    T, kw = int(p["cu"][-1]), p["kw"]
    q, k = (p[n].reshape(T, hk, dk).repeat_interleave(h // hk, 1) for n in ("q", "k"))
    g = p["g"].reshape(T, h, 1).expand(T, h, dk)
    dt = kw.get("dt_bias")
    return oracle.Problem(q, k, p["v"].reshape(T, h, -1), g, p["beta"].reshape(T, h), cu_seqlens=p["cu"], scale=kw["scale"],
                          eps=EPS, a_log=kw.get("a_log"), dt_bias=None if dt is None else dt[:, None].expand(h, dk),
                          l2norm=kw.get("l2norm_qk", True), beta_sigmoid=kw.get("beta_sigmoid", False),
                          gate_in_kernel=kw.get("gate_in_kernel", False))


def cuda(x):
    if isinstance(x, dict):
        return {n: cuda(v) for n, v in x.items()}
    return x.cuda() if isinstance(x, torch.Tensor) else x


def off(got, ref):
    """Relative 2-norm of the difference; the finite result is asked for too."""
    x = got.detach().double().cpu().numpy().reshape(np.shape(ref))
    assert np.all(np.isfinite(x))
    den = np.linalg.norm(ref)
    return float(np.linalg.norm(x - ref) / den) if den else float(np.linalg.norm(x))


def check(got, ref, what, tol=None):
    e, tol = off(got, ref), TOL[got.dtype] if tol is None else tol
    # below 2^-126 fp32 has no relative precision left (and below 2^-149 nothing but zero): each value may be
    # off by that much, the 2-norm of n of them by sqrt(n) 2^-126
    norm = np.linalg.norm(ref)
    if norm > 0:
        tol += np.sqrt(np.size(ref)) * 2.0 ** -126 / norm
    assert e <= tol, f"{what}: off by {e:.3g} of its norm, at most {tol:.3g} is wanted"
    return e


def args(p):
    return p["q"], p["k"], p["v"], p["g"], p["beta"]
