"""Gradients of the gated delta rule with one gate per head on the GPU: against the 64-bit oracle's and against
differences of the forward's oracle."""
import numpy as np
import pytest
import torch

import oracle
from gdn_testutil import args, check, cuda, oracle_of, problem

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _bwd(kda, p, d_out=True, d_final=True, **kw):
    d = cuda(p)
    got = kda.kda_gdn_chunk_bwd(*args(d), d["d_out"] if d_out else None, d_final_state=d["d_final"] if d_final else None,
                                want_d_initial_state=True, **dict(d["kw"], **kw))
    torch.cuda.synchronize()
    return got


def _reference(p, d_out=True, d_final=True):
    """The oracle's gradients, summed over what one gate or one key head stands for."""
    r = oracle.chunk_bwd(oracle_of(p), p["kw"]["initial_state"], p["d_out"] if d_out else None, p["d_final"] if d_final else None)
    h, hk = p["v"].shape[-2], p["q"].shape[-2]
    for n in ("dq", "dk"):
        r[n] = r[n].reshape(-1, hk, h // hk, r[n].shape[-1]).sum(2)
    r["dg"], r["ddt_bias"] = r["dg"].sum(-1), r["ddt_bias"].sum(-1)
    r["d_initial_state"] = r["d_initial"]
    return r


def _check_bwd(kda, p, **which):
    got, ref = _bwd(kda, p, **which), _reference(p, **which)
    for n in ("dq", "dk", "dv", "dg", "dbeta", "d_initial_state"):
        check(got[n], ref[n], n)
    for n in ("da_log", "ddt_bias"):
        if p["kw"].get("gate_in_kernel"):
            # a sum over all tokens, whose signs differ: held to the size of what is summed
            size = np.sqrt((ref["dg"].reshape(-1, ref["da_log"].shape[0]) ** 2).sum(0))
            off = np.abs(got[n].double().cpu().numpy() - ref[n])
            assert np.all(off <= 7e-6 * (np.abs(ref[n]) + size)), n
        else:
            assert got[n] is None


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (64, 128), (128, 64)])
@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 130])
def test_bwd_lengths(cuda_lib, dtype, dk, dv, T):
    _check_bwd(cuda_lib, problem([T, T], dk=dk, dv=dv, dtype=dtype, seed=T + dk, initial=T != 2))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("gate", ["slow", "strong"])
@pytest.mark.parametrize("raw", [False, True])
def test_bwd_gates(cuda_lib, dtype, gate, raw):
    _check_bwd(cuda_lib, problem([333], dtype=dtype, gate=gate, raw=raw, seed=7))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("hk,h", [(1, 1), (1, 5), (3, 6), (4, 4)])
def test_bwd_packed(cuda_lib, dtype, hk, h):
    _check_bwd(cuda_lib, problem([0, 1, 64, 129, 0, 200, 3, 0], hk=hk, h=h, dtype=dtype, seed=h))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("which", [dict(d_out=False), dict(d_final=False)])
def test_bwd_one_gradient_given(cuda_lib, dtype, which):
    _check_bwd(cuda_lib, problem([200], dtype=dtype, seed=3), **which)


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_bwd_many_heads(cuda_lib, dtype, dk, dv):
    """More chains than half the SMs (a CTA has all 128 value channels) of many chunks."""
    _check_bwd(cuda_lib, problem([600, 0, 1, 577, 64, 128, 129, 640, 63, 511, 90, 7], hk=4, h=8, dk=dk, dv=dv, dtype=dtype, seed=dk))


def test_bwd_long(cuda_lib):
    _check_bwd(cuda_lib, problem([2048], hk=1, h=2, seed=3))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("what", ["beta 0", "no decay", "decay to zero", "zero keys", "loss on few tokens", "huge values"])
def test_bwd_corners(cuda_lib, what, dtype):
    p = problem([150], hk=1, h=2, dtype=dtype, raw=True, seed=11)
    p["kw"]["l2norm_qk"] = True
    if what == "beta 0":
        p["beta"][:, 20:90] = 0
    elif what == "no decay":
        p["g"][:] = 0
    elif what == "decay to zero":
        p["g"][:, ::7] = -200.0
    elif what == "zero keys":
        p["k"][:, 10:30] = 0
    elif what == "loss on few tokens":
        p["d_out"][:, :100] = 0
        p["d_out"][:, 101:] = 0
    else:
        p["v"] = (p["v"].float() * 1e20).to(dtype)
        p["d_out"] = (p["d_out"].float() * 1e-25).to(dtype)
        p["d_final"] *= 1e-25
    _check_bwd(cuda_lib, p)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_bwd_layouts_are_the_same_numbers(cuda_lib, dtype):
    for lens in ([130, 130], [70, 0, 65]):
        p = problem(lens, dk=64, dtype=dtype, seed=5, packed=len(set(lens)) > 1)
        want = _bwd(cuda_lib, p)
        flip = lambda x: x.transpose(-1, -2).contiguous()  # noqa: E731
        got = _bwd(cuda_lib, dict(p, d_final=flip(p["d_final"]), kw=dict(p["kw"], initial_state=flip(p["kw"]["initial_state"]))),
                   state_v_first=True)
        got["d_initial_state"] = got["d_initial_state"].transpose(-1, -2)
        for n in want:
            assert torch.equal(got[n], want[n]), n
        axis = 2 if p["q"].dim() == 4 else 1
        hm = dict(p, **{n: p[n].transpose(axis - 1, axis).contiguous() for n in ("q", "k", "v", "g", "beta", "d_out")})
        got = _bwd(cuda_lib, hm, head_major=True)
        for n in ("dq", "dk", "dv", "dg", "dbeta"):
            got[n] = got[n].transpose(axis - 1, axis)
        for n in want:
            assert torch.equal(got[n], want[n]), n


def test_bwd_is_the_same_each_time(cuda_lib):
    p = problem([500, 77], seed=1)
    a, b = _bwd(cuda_lib, p), _bwd(cuda_lib, p)
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_bwd_no_tokens(cuda_lib):
    p = problem([0, 0], packed=True)
    got = _bwd(cuda_lib, p)
    assert torch.equal(got["d_initial_state"].cpu(), p["d_final"])
    assert float(got["da_log"].abs().max()) == 0 and float(got["ddt_bias"].abs().max()) == 0


def test_bwd_against_differences(cuda_lib):
    """Central differences of the forward's 64-bit oracle along one direction a tensor; the third derivative's term is
    below 1e-6 of the slope at this step, so the tolerance is the gradients' own."""
    p = problem([70], hk=1, h=2, dtype=F32, seed=8)
    got = _bwd(cuda_lib, p)
    gen = torch.Generator().manual_seed(0)
    step = 1e-4

    def loss(q):
        o, f = oracle.chunk_fwd(oracle_of(q), q["kw"]["initial_state"])
        return (o * p["d_out"].double().numpy().reshape(o.shape)).sum() + (f * p["d_final"].double().numpy()).sum()
    for n, key in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dg"), ("beta", "dbeta"), ("initial_state", "d_initial_state"),
                   ("a_log", "da_log"), ("dt_bias", "ddt_bias")):
        inside = n in p["kw"]
        x = (p["kw"] if inside else p)[n].double()
        u = torch.randn(x.shape, generator=gen, dtype=torch.float64)
        sides = []
        for s in (step, -step):
            q = dict(p, kw=dict(p["kw"]))
            (q["kw"] if inside else q)[n] = x + s * u
            sides.append(loss(q))
        slope, mine = (sides[0] - sides[1]) / (2 * step), float((got[key].double().cpu() * u).sum())
        size = float(got[key].double().norm()) * float(u.norm()) / u.numel() ** 0.5
        assert abs(slope - mine) <= 2e-5 * (abs(slope) + size), (n, slope, mine)
