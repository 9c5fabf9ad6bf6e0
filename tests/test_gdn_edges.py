"""The gated delta rule with one gate per head where its numbers leave the ordinary range, on the GPU against the 64-bit
oracle."""
import numpy as np
import pytest
import torch

import oracle
from gdn_testutil import args, check, cuda, oracle_of, problem
from test_gdn_bwd import _reference

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _check_both(kda, p, eps=None):
    """Forward and backward; eps: of the norms, if not the test problems' own."""
    d = cuda(p)
    kw = dict(d["kw"]) if eps is None else dict(d["kw"], eps=eps)
    out, fin = kda.kda_gdn_chunk_fwd(*args(d), **kw)
    o, f = oracle.chunk_fwd(oracle_of(p), p["kw"]["initial_state"])
    check(out, o, "o")
    check(fin, f, "final state")
    got = kda.kda_gdn_chunk_bwd(*args(d), d["d_out"], d_final_state=d["d_final"], want_d_initial_state=True, **kw)
    ref = _reference(p)
    for n in ("dq", "dk", "dv", "dg", "dbeta", "d_initial_state"):
        check(got[n], ref[n], n)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dk", [64, 128])
@pytest.mark.parametrize("lens", [[1], [63], [65, 65], [130, 0, 7]])
def test_norms_without_eps(cuda_lib, dtype, dk, lens):
    """eps = 0: what fills a chunk behind a sequence's end has no norm to divide by.  (The oracle's eps of 1e-6 is 2e-8
    of these rows' sums of squares, below 64, and less of what follows: far inside the tolerance.)"""
    _check_both(cuda_lib, problem(lens, dk=dk, dtype=dtype, seed=sum(lens)), eps=0.0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("l2", [True, False])
@pytest.mark.parametrize("k,q", [(1e-25, 1.0), (1e-35, 1.0), (1.0, 1e-25), (1e-25, 1e-25), (1e-25, 1e22), (1e-30, 1e30)])
def test_keys_and_queries_whose_squares_leave_the_range(cuda_lib, dtype, l2, k, q):
    """A chunk's keys or queries of a size whose squares fp32 cannot hold: the unit of q k^T's pieces still fits.  (The
    middle chunk's alone; q is not normalised where its squares are infinite in fp32.)"""
    p = problem([180], hk=1, h=2, dtype=dtype, raw=True, seed=12, initial=False)
    p["kw"]["l2norm_qk"] = l2 and q <= 1
    for n, size in (("k", k), ("q", q)):
        p[n][:, 64:128] = (p[n][:, 64:128].float() * size).to(dtype)
    d = cuda(p)
    out, fin = cuda_lib.kda_gdn_chunk_fwd(*args(d), **d["kw"])
    o, f = oracle.chunk_fwd(oracle_of(p), None)
    check(fin, f, "final state")
    o, got = o.reshape(180, 2, -1), out.reshape(180, 2, -1)
    for r in (slice(0, 64), slice(64, 128), slice(128, 180)):
        check(got[r], o[r], f"o of tokens {r}")
    got, ref = cuda_lib.kda_gdn_chunk_bwd(*args(d), d["d_out"], d_final_state=d["d_final"], **d["kw"]), _reference(p)
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        check(got[n], ref[n], n)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lens", [[70, 33], [0, 0], [3] * 1100])
@pytest.mark.parametrize("head_major", [False, True])
def test_padding_behind_the_last_sequence(cuda_lib, dtype, lens, head_major):
    """What lies there may hold anything: it is not read, and what the call allocates is zero there."""
    p, pad = problem(lens, hk=1, h=3, dk=64, dv=64, dtype=dtype, packed=True, seed=len(lens)), 77
    want = cuda_lib.kda_gdn_chunk_fwd(*args(cuda(p)), **cuda(p["kw"]))[0] if sum(lens) else p["v"].cuda()
    wants = cuda_lib.kda_gdn_chunk_bwd(*args(cuda(p)), p["d_out"].cuda(), d_final_state=p["d_final"].cuda(), **cuda(p["kw"]))
    for n in ("q", "k", "v", "g", "beta", "d_out"):
        p[n] = torch.cat([p[n], torch.full((pad, *p[n].shape[1:]), float("nan"), dtype=p[n].dtype)])
        if head_major:
            p[n] = p[n].transpose(0, 1).contiguous()
    d = cuda(p)
    for _ in range(2):  # what the allocator hands out next held NaN
        for n in ("q", "k", "v", "g", "beta"):
            torch.full_like(d[n], float("nan"))
    out = cuda_lib.kda_gdn_chunk_fwd(*args(d), head_major=head_major, **d["kw"])[0]
    got = dict(cuda_lib.kda_gdn_chunk_bwd(*args(d), d["d_out"], d_final_state=d["d_final"], head_major=head_major, **d["kw"]), out=out)
    for n in ("out", "dq", "dk", "dv", "dg", "dbeta"):
        x = got[n].transpose(0, 1) if head_major else got[n]
        assert torch.equal(x[:sum(lens)], want if n == "out" else wants[n]), n
        assert bool((x[sum(lens):] == 0).all()), n
    for n in ("da_log", "ddt_bias", "d_initial_state"):
        assert torch.equal(got[n], wants[n]), n


@pytest.mark.parametrize("dtype,dk", [(BF16, 128), (BF16, 64), (F32, 64), (F32, 128)])
@pytest.mark.parametrize("T", [64, 65, 130, 1093])
def test_results_do_not_depend_on_what_else_is_computed(cuda_lib, dtype, dk, T):
    """Many chains (a CTA has all 128 value channels, in two groups of warps) and a few of the same ones (a CTA has half
    of them): a warp's arithmetic is its own, so the bits are the same."""
    h = 80
    p = problem([T, T], hk=h, h=h, dk=dk, dtype=dtype, seed=T)
    few = dict(p, **{n: p[n][:1, :, 3:5].contiguous() for n in ("q", "k", "v", "g", "beta", "d_out")}, d_final=p["d_final"][:1, 3:5].contiguous())
    few["kw"] = dict(p["kw"], a_log=p["kw"]["a_log"][3:5].contiguous(), dt_bias=p["kw"]["dt_bias"][3:5].contiguous(),
                     initial_state=p["kw"]["initial_state"][:1, 3:5].contiguous())
    res = []
    for x in (p, few):
        d = cuda(x)
        res.append((*cuda_lib.kda_gdn_chunk_fwd(*args(d), **d["kw"]),
                    cuda_lib.kda_gdn_chunk_bwd(*args(d), d["d_out"], d_final_state=d["d_final"], **d["kw"])))
    (out, fin, g), (out1, fin1, g1) = res
    assert torch.equal(out[:1, :, 3:5], out1) and torch.equal(fin[:1, 3:5], fin1)
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        assert torch.equal(g[n][:1, :, 3:5], g1[n]), n
    assert torch.equal(g["d_initial_state"][:1, 3:5], g1["d_initial_state"])
