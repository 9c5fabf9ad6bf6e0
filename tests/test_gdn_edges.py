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
