"""The gated delta rule with one gate per head where its numbers leave the ordinary range, on the GPU against the 64-bit
oracle."""
import numpy as np
import pytest
import torch

import oracle
from gdn_testutil import TOL, args, check, cuda, oracle_of, problem
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


def _per_token(got, ref, T, h):
    """2-norms over the channels of the error and of the result, for each token and head."""
    ref = np.asarray(ref).reshape(T, h, -1)
    x = got.double().cpu().numpy().reshape(ref.shape)
    return np.linalg.norm(x - ref, axis=-1), np.linalg.norm(ref, axis=-1)


# As gdn_testutil's, but fp32's four products in a row with errors that are independent, so that their squares add:
# sqrt(4) / 4 of their sum
TOKEN_TOL = {BF16: TOL[BF16], F32: TOL[F32] / 2}


def _all(kda, p):
    d = cuda(p)
    out, fin = kda.kda_gdn_chunk_fwd(*args(d), **d["kw"])
    got = kda.kda_gdn_chunk_bwd(*args(d), d["d_out"], d_final_state=d["d_final"], want_d_initial_state=True, **d["kw"])
    o, f = oracle.chunk_fwd(oracle_of(p), p["kw"]["initial_state"])
    return dict(got, out=out, final=fin), dict(_reference(p), out=o, final=f)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("gate", ["slow", "strong"])
@pytest.mark.parametrize("lens", [[300], [1, 130, 0, 70, 2]])
def test_every_token_and_head_by_itself(cuda_lib, dtype, gate, lens):
    """No token, head or sequence hides behind the others' size.  A token's sum may cancel (dq of two value heads whose
    states have decayed is (c1 + c2) k with numbers c of either sign), its terms are then of the size of its neighbours'
    results: errors of 2^-12 of terms a hundred times the sum are 2^-5 of the sum.  So a token is held to its own size and
    the root mean square of its head's tokens, which no sum over tokens dilutes.  dg and dbeta are one number: a dot
    product of 128 channels, which d_final makes larger at the sequences' last tokens than elsewhere (its k dS is 0.1
    sqrt(128) beside P dO's 0.09 k.q / |k||q| sqrt(128): ten times).  Where such a one cancels its terms are still of that
    size, so these are held to the largest of their head in the mean square's place."""
    p = problem(lens, hk=2, h=4, dtype=dtype, gate=gate, seed=21)
    got, ref = _all(cuda_lib, p)
    T = sum(lens)
    for n, h in (("out", 4), ("dq", 2), ("dk", 2), ("dv", 4), ("dg", 4), ("dbeta", 4)):
        e, size = _per_token(got[n], ref[n], T, h)
        number = n in ("dg", "dbeta")
        bound = TOKEN_TOL[F32 if number else dtype] * (size + (size.max(0) if number else np.sqrt((size ** 2).mean(0))))
        assert np.all(e <= bound), (n, np.max(e / bound))
    for n in ("final", "d_initial_state"):
        r = np.asarray(ref[n]).reshape(len(lens), 4, -1)
        e = np.linalg.norm(got[n].double().cpu().numpy().reshape(r.shape) - r, axis=-1)
        assert np.all(e <= TOKEN_TOL[F32] * np.linalg.norm(r, axis=-1)), n


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("what", ["q", "d_out", "v"])
def test_tokens_of_very_different_size_in_one_chunk(cuda_lib, dtype, what):
    """Tokens of 1, 2^-20 and 2^-30 beside each other.  dq where d_out differs is a token's own and keeps its own
    accuracy.  P (out where q differs, here without norms) is held against its chunk's largest: its pieces end 2^-15
    below an ordinary error of that, and that largest is a bound from norms, by Gaussian rows' sqrt(128) = 2^3.5 too high:
    2^-11 with sums of two terms.  What sums over a chunk's tokens is as good as its largest."""
    T = 192
    p = problem([T], hk=1, h=2, dtype=dtype, raw=what == "q", seed=5)
    e = torch.tensor([0, -20, -30])[torch.randint(0, 3, (T,), generator=torch.Generator().manual_seed(9))]
    p[what] = (p[what].float() * (2.0 ** e).view(1, T, 1, 1)).to(dtype)
    p["d_final"] *= 0  # a gradient of the last state would reach every token
    if what == "v":
        p["kw"]["initial_state"] *= 0
    got, ref = _all(cuda_lib, p)
    share = {("out", "q"): 2.0 ** -11, ("dq", "d_out"): 0.0}
    for n, h in (("out", 2), ("dq", 1), ("dk", 1), ("dv", 2), ("dg", 2), ("dbeta", 2)):
        err, size = _per_token(got[n], ref[n], T, h)
        most = np.repeat(size.reshape(T // 64, 64, h).max(1), 64, 0)
        tol = TOKEN_TOL[dtype if n not in ("dg", "dbeta") else F32]
        bound = tol * (size + share.get((n, what), 1.0) * most)
        assert np.all(err <= bound), (n, np.max(err / bound))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dv", [64, 128])
def test_step_result_in_the_values_place(cuda_lib, dtype, dv):
    d = cuda(problem([3] * 40, hk=2, h=4, dv=dv, dtype=dtype, packed=False, seed=8))
    kw = {n: v for n, v in d["kw"].items() if n not in ("initial_state", "cu_seqlens")}
    pool, idx = 0.1 * torch.randn(40, 4, 128, dv, device="cuda"), torch.arange(40, device="cuda").flip(0).contiguous()
    mine = pool.clone()
    want = cuda_lib.kda_gdn_recurrent_step(*args(d), pool, idx, **kw)
    got = cuda_lib.kda_gdn_recurrent_step(*args(d), mine, idx, out=d["v"], **kw)
    assert got is d["v"] and torch.equal(got, want) and torch.equal(mine, pool)
