"""The gated delta rule with one gate per head on the GPU against the 64-bit oracle: chunked forward, and the recurrent
step on pool states."""
import numpy as np
import pytest
import torch

import oracle
from gdn_testutil import TOL, args, check, cuda, off, oracle_of, problem

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _fwd(kda, p, **kw):
    d = cuda(p)
    got = kda.kda_gdn_chunk_fwd(*args(d), **dict(d["kw"], **kw))
    torch.cuda.synchronize()
    return got


def _check_fwd(kda, p):
    out, fin = _fwd(kda, p)
    o, f = oracle.chunk_fwd(oracle_of(p), p["kw"]["initial_state"])
    check(out, o, "o")
    check(fin, f, "final state")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (64, 128), (128, 64)])
@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 130])
def test_fwd_lengths(cuda_lib, dtype, dk, dv, T):
    _check_fwd(cuda_lib, problem([T, T], dk=dk, dv=dv, dtype=dtype, seed=T + dk, initial=T != 2))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("gate", ["slow", "strong"])
@pytest.mark.parametrize("raw", [False, True])
def test_fwd_gates(cuda_lib, dtype, gate, raw):
    _check_fwd(cuda_lib, problem([333], dtype=dtype, gate=gate, raw=raw, seed=7))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("hk,h", [(1, 1), (1, 5), (3, 6), (4, 4)])
def test_fwd_packed(cuda_lib, dtype, hk, h):
    _check_fwd(cuda_lib, problem([0, 1, 64, 129, 0, 200, 3, 0], hk=hk, h=h, dtype=dtype, seed=h))


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_fwd_many_heads(cuda_lib, dtype, dk, dv):
    """More chains than half the SMs (a CTA has all 128 value channels) of many chunks."""
    _check_fwd(cuda_lib, problem([600, 0, 1, 577, 64, 128, 129, 640, 63, 511, 90, 7], hk=4, h=8, dk=dk, dv=dv, dtype=dtype, seed=dk))


def test_more_packed_sequences_than_are_ordered(cuda_lib):
    _check_fwd(cuda_lib, problem([1, 0, 2] * 400, hk=1, h=1, dk=64, dv=64, seed=2))


def test_tokens_behind_the_last_sequence_are_left_alone(cuda_lib):
    p = problem([70, 33], seed=3)
    want = _fwd(cuda_lib, p)
    d = cuda(p)
    for n in ("q", "k", "v", "g", "beta"):  # what is not read may hold anything
        d[n] = torch.cat([d[n], torch.full_like(d[n][:50], float("nan"))])
    out = torch.full_like(d["v"], 7.0)
    got = cuda_lib.kda_gdn_chunk_fwd(*args(d), **dict(d["kw"], out=out))
    assert torch.equal(got[0][:103], want[0]) and torch.equal(got[1], want[1]) and bool((out[103:] == 7).all())


def test_fwd_long(cuda_lib):
    _check_fwd(cuda_lib, problem([4096], hk=1, h=2, seed=3))


@pytest.mark.parametrize("what", ["beta 0", "no decay", "decay to zero", "zero keys", "equal keys", "huge values", "tiny values"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_fwd_corners(cuda_lib, what, dtype):
    p = problem([150], hk=1, h=2, dtype=dtype, raw=True, seed=11)
    p["kw"]["l2norm_qk"] = True
    if what == "beta 0":
        p["beta"][:, 20:90] = 0
    elif what == "no decay":
        p["g"][:] = 0
    elif what == "decay to zero":
        p["g"][:, ::7] = -200.0
        p["g"][:, 64] = -float("inf")
    elif what == "zero keys":
        p["k"][:, 10:30] = 0
        p["q"][:, 5] = 0
    elif what == "equal keys":  # the strongest coupling inside a chunk
        p["k"][:] = p["k"][:, :1]
        p["beta"][:] = 1
    elif what == "huge values":
        p["v"] = (p["v"].float() * 1e30).to(dtype)
    else:
        p["v"] = (p["v"].float() * 1e-30).to(dtype)
        p["kw"]["initial_state"] *= 1e-30
    _check_fwd(cuda_lib, p)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_fwd_layouts_are_the_same_numbers(cuda_lib, dtype):
    for lens in ([130, 130], [70, 0, 65]):
        p = problem(lens, dv=64, dtype=dtype, seed=5, packed=len(set(lens)) > 1)
        out, fin = _fwd(cuda_lib, p)
        vf = dict(p, kw=dict(p["kw"], initial_state=p["kw"]["initial_state"].transpose(-1, -2).contiguous()))
        out2, fin2 = _fwd(cuda_lib, vf, state_v_first=True)
        assert torch.equal(out, out2) and torch.equal(fin, fin2.transpose(-1, -2))
        hm = dict(p)
        for n in ("q", "k", "v", "g", "beta"):
            axis = 2 if p["q"].dim() == 4 else 1
            hm[n] = p[n].transpose(axis - 1, axis).contiguous()
        out3, fin3 = _fwd(cuda_lib, hm, head_major=True)
        assert torch.equal(out, out3.transpose(-3, -2)) and torch.equal(fin, fin3)


def test_fwd_in_place_state_and_given_buffers(cuda_lib):
    p = problem([100, 37], seed=9)
    out, fin = _fwd(cuda_lib, p)
    d = cuda(p)
    state, mine = d["kw"]["initial_state"], torch.empty_like(d["v"])
    got, got_fin = cuda_lib.kda_gdn_chunk_fwd(*args(d), **dict(d["kw"], final_state=state, out=mine))
    assert got is mine and got_fin is state and torch.equal(mine, out) and torch.equal(state, fin)
    none = cuda_lib.kda_gdn_chunk_fwd(*args(d), **dict(cuda(p)["kw"], output_final_state=False))
    assert none[1] is None and torch.equal(none[0], out)


def test_fwd_no_tokens(cuda_lib):
    p = problem([0, 0], packed=True)
    out, fin = _fwd(cuda_lib, p)
    assert out.numel() == 0 and torch.equal(fin.cpu(), p["kw"]["initial_state"])
    p = problem([0], packed=False, initial=False)
    assert float(_fwd(cuda_lib, p)[1].abs().max()) == 0


def test_fwd_nan_stays_in_its_sequence(cuda_lib):
    p = problem([90, 70, 64], seed=2)
    want = _fwd(cuda_lib, p)
    p["v"][100, 1, 3] = float("nan")
    got = _fwd(cuda_lib, p)
    assert torch.isnan(got[0][100, 1, 3])
    for a, b in ((0, 90), (160, 224)):
        assert torch.equal(got[0][a:b], want[0][a:b])
    assert torch.equal(got[1][[0, 2]], want[1][[0, 2]])


@pytest.mark.parametrize("dtype,cache", [(BF16, F32), (BF16, BF16), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (64, 128), (128, 64)])
@pytest.mark.parametrize("T,gap,v_first", [(1, 0, False), (3, 3, False), (2, 5, True)])
def test_step(cuda_lib, dtype, cache, dk, dv, T, gap, v_first):
    N, h, rows = 6, 4, 9
    p = problem([T] * N, hk=2, h=h, dk=dk, dv=dv, dtype=dtype, packed=False, seed=T + dv)
    base = (0.1 * torch.randn(rows, h * dk * dv + gap, generator=torch.Generator().manual_seed(1))).to(cache).cuda()
    before = base.clone()
    pool = base[:, :h * dk * dv].view(rows, h, *((dv, dk) if v_first else (dk, dv)))
    idx, flags = torch.tensor([4, -1, 0, 9, 7, 2]), torch.tensor([True, True, False, True, True, True])
    S0 = torch.zeros(N, h, dk, dv, dtype=torch.float64)
    for i, r in enumerate(idx.tolist()):
        if 0 <= r < rows and flags[i]:
            S0[i] = (pool[r].transpose(-1, -2) if v_first else pool[r]).double().cpu()
    d = cuda(p)
    kw = {n: v for n, v in d["kw"].items() if n not in ("initial_state", "cu_seqlens")}
    out = cuda_lib.kda_gdn_recurrent_step(*args(d), pool, idx.cuda().to(torch.int32 if gap else torch.int64), flags.cuda(),
                                          state_v_first=v_first, **kw)
    o, f = oracle.chunk_fwd(oracle_of(p), S0)
    check(out, o, "o")
    for i, r in enumerate(idx.tolist()):
        if 0 <= r < rows:
            check(pool[r].transpose(-1, -2) if v_first else pool[r], f[i], f"row {r}")
    others = [r for r in range(rows) if r not in idx.tolist()]
    assert torch.equal(base[others], before[others])
    assert torch.equal(base[:, h * dk * dv:], before[:, h * dk * dv:])


def test_offsets_beyond_32_bits(cuda_lib):
    """2.2 G elements of v and out, and a pool of as many: a run cut at a chunk's end gives the same bits, and the step
    finds the last row."""
    T, cut, H, D = 262_208 + 77, 262_144, 64, 128
    gen = torch.Generator(device="cuda").manual_seed(0)
    q, k = (torch.randn(1, T, 1, D, generator=gen, device="cuda").bfloat16() for _ in range(2))
    v = torch.empty(1, T, H, D, dtype=BF16, device="cuda").normal_(generator=gen)
    g, beta = (torch.randn(1, T, H, generator=gen, device="cuda") for _ in range(2))
    kw = dict(a_log=torch.zeros(H, device="cuda"), gate_in_kernel=True, beta_sigmoid=True)
    out, fin = cuda_lib.kda_gdn_chunk_fwd(q, k, v, g, beta, **kw)
    _, mid = cuda_lib.kda_gdn_chunk_fwd(*(x[:, :cut].contiguous() for x in (q, k, v, g, beta)), **kw)
    end = [x[:, cut:].contiguous() for x in (q, k, v, g, beta)]
    late, last = cuda_lib.kda_gdn_chunk_fwd(*end, initial_state=mid, **kw)
    assert torch.equal(out[:, cut:], late) and torch.equal(fin, last)
    del v, out, late
    pool = torch.zeros(2100, H, D, D, device="cuda")  # 2.2 G elements
    pool[2099] = mid[0]
    idx = torch.tensor([2099], device="cuda")
    one = cuda_lib.kda_gdn_recurrent_step(*(x[:, :1].contiguous() for x in end), pool, idx, **kw)
    want, state = cuda_lib.kda_gdn_chunk_fwd(*(x[:, :1].contiguous() for x in end), initial_state=mid, **kw)
    assert off(one, want.double().cpu().numpy()) <= 2 * TOL[BF16] and off(pool[2099], state[0].double().cpu().numpy()) <= 2 * TOL[F32]
    assert float(pool[:2099].abs().max()) == 0


def test_prefill_then_decode_is_one_run(cuda_lib):
    """The chunked call on a prefix and the step on what follows, against the oracle on all of it."""
    p = problem([140], hk=2, h=4, seed=4)
    d = cuda(p)
    cut = 133
    out, fin = cuda_lib.kda_gdn_chunk_fwd(*(x[:, :cut].contiguous() for x in args(d)), **d["kw"])
    pool = torch.zeros(3, *fin.shape[1:], device="cuda")
    pool[2] = fin[0]
    kw = {n: v for n, v in d["kw"].items() if n not in ("initial_state", "cu_seqlens")}
    idx = torch.tensor([2], dtype=torch.int32, device="cuda")
    parts = [out]
    for t in range(cut, 140):
        parts.append(cuda_lib.kda_gdn_recurrent_step(*(x[:, t:t + 1].contiguous() for x in args(d)), pool, idx, **kw))
    o, f = oracle.chunk_fwd(oracle_of(p), p["kw"]["initial_state"])
    check(torch.cat(parts, 1), o, "o")
    check(pool[2], f[0], "state")


def test_equals_the_per_channel_rule(cuda_lib):
    """kda_chunk_fwd with the gate repeated over the channels, in fp32 (its own tolerance: 1e-4 of the largest)."""
    p = problem([200], hk=2, h=4, dtype=F32, seed=6)
    d = cuda(p)
    out, fin = _fwd(cuda_lib, p)
    kw = dict(d["kw"], dt_bias=d["kw"]["dt_bias"][:, None].expand(-1, 128).contiguous())
    o, f = cuda_lib.kda_chunk_fwd(d["q"], d["k"], d["v"], d["g"][..., None].expand(*d["g"].shape, 128).contiguous(), d["beta"], **kw)
    assert float((out - o).abs().max()) <= 1.1e-4 * float(o.abs().max())
    assert float((fin - f).abs().max()) <= 1.1e-4 * float(f.abs().max())
