"""Low-rank adapters of many requests on the GPU against 64-bit arithmetic: results, gradients, rows and adapters that
nothing is to happen to, and the calls around the shared 8-bit projection.

Tolerances, relative to the 2-norm of the result:
  bf16  one rounding, at most half a step: 2^-8, and u to 16 bits: below 2^-8 + 2^-15
  fp32  operands of 24 bits; a tensor-core step drops less than 2^-23 of its running sum, which is taken into
        registers after at most 8 steps of k with 6 products each; two products in a row:
        2 * 48 * 2^-23 = 1.2e-5 if every error had one sign; they do not, half of that is asked for
"""
import numpy as np
import pytest
import torch

from gdn_testutil import off

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
TOL = {BF16: 2.0 ** -8 + 2.0 ** -15, F32: 6e-6}


def problem(lens, n_in, n_out, rank, adapters=3, dtype=BF16, packed=True, tail=0, seed=0, idx=None, idx_dtype=torch.int32):
    gen = torch.Generator().manual_seed(seed)

    def randn(*s):
        return torch.randn(*s, generator=gen)
    rows = sum(lens) + tail
    p = dict(x=randn(rows, n_in).to(dtype), a=(randn(adapters, rank, n_in) * n_in ** -0.5).to(dtype),
             b=(randn(adapters, n_out, rank) * rank ** -0.5).to(dtype), y=randn(rows, n_out).to(dtype),
             d_out=randn(rows, n_out).to(dtype), d_x=randn(rows, n_in).to(dtype), scale=0.5 + torch.rand(adapters, generator=gen))
    p["idx"] = torch.randint(-1, adapters + 1, (len(lens),), generator=gen).to(idx_dtype) if idx is None else torch.tensor(idx, dtype=idx_dtype)
    cu = np.concatenate([[0], np.cumsum(lens)])
    p["cu"] = torch.tensor(cu, dtype=torch.int32) if packed else None
    p["spans"] = [(int(cu[i]), int(cu[i + 1]), l) for i, l in enumerate(p["idx"].tolist()) if 0 <= l < adapters]
    return p


def reference(p):
    f = {n: p[n].double() for n in ("x", "a", "b", "y", "d_out", "d_x", "scale")}
    out, dx, da, db = f["y"].clone(), f["d_x"].clone(), torch.zeros_like(f["a"]), torch.zeros_like(f["b"])
    for r0, r1, l in p["spans"]:
        x, d, s = f["x"][r0:r1], f["d_out"][r0:r1], f["scale"][l]
        out[r0:r1] += s * (x @ f["a"][l].t()) @ f["b"][l].t()
        du = s * d @ f["b"][l]
        dx[r0:r1] += du @ f["a"][l]
        da[l] += du.t() @ x
        db[l] += s * d.t() @ (x @ f["a"][l].t())
    return [t.numpy() for t in (out, dx, da, db)]


def cuda(p):
    return {n: v.cuda() if isinstance(v, torch.Tensor) else v for n, v in p.items()}


def forward(kda, p, **kw):
    d = cuda(p)
    return kda.kda_lora(d["x"], d["a"], d["b"], d["idx"], d["y"], cu_seqlens=d["cu"], scale=d["scale"], **kw)


def backward(kda, p, **kw):
    d = cuda(p)
    return kda.kda_lora_bwd(d["d_out"], d["x"], d["a"], d["b"], d["idx"], d["d_x"], cu_seqlens=d["cu"], scale=d["scale"], **kw)


def check(p, got, ref):
    for name, g, r in zip(("out", "dx", "da", "db"), got, ref):
        if g is not None:
            e = off(g, r)
            assert e <= TOL[g.dtype], f"{name}: off by {e:.3g}, at most {TOL[g.dtype]:.3g} is wanted"


def run(kda, p):
    check(p, [forward(kda, p), *backward(kda, p)], reference(p))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rank", [1, 3, 8, 16, 17, 24, 32, 60, 64, 100, 128])
def test_ranks(cuda_lib, dtype, rank):
    run(cuda_lib, problem([5, 0, 70, 64, 1], 256, 320, rank, dtype=dtype, idx=[2, 1, 0, 2, 3], seed=rank))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n_in,n_out", [(1, 1), (8, 4), (33, 31), (100, 200), (1000, 36), (777, 1111), (64, 4196), (4100, 8)])
def test_widths(cuda_lib, dtype, n_in, n_out):
    run(cuda_lib, problem([17, 65, 40], n_in, n_out, 12, dtype=dtype, idx=[0, 1, 0], seed=n_in))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows", [1, 2, 16, 17, 64, 65, 130])
@pytest.mark.parametrize("requests", [1, 5])
def test_equal_requests(cuda_lib, dtype, rows, requests):
    run(cuda_lib, problem([rows] * requests, 512, 264, 16, dtype=dtype, packed=False, seed=rows, idx_dtype=torch.int64))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rank", [30, 50, 128])
def test_ranks_of_few_rows_each(cuda_lib, dtype, rank):
    run(cuda_lib, problem([1] * 20, 520, 300, rank, dtype=dtype, packed=False, seed=rank))
    run(cuda_lib, problem([3, 40, 0, 1, 1, 2, 1, 1], 260, 130, rank, dtype=dtype, seed=rank))


def test_offsets_beyond_32_bits(cuda_lib):
    """2.3 G elements of y: the last request's rows against a call on them alone."""
    rows, n_out = 70_001, 32_768
    gen = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(rows, 64, generator=gen, device="cuda").bfloat16()
    a, b = (torch.randn(*s, generator=gen, device="cuda").bfloat16() for s in ((2, 8, 64), (2, n_out, 8)))
    y = torch.zeros(rows, n_out, dtype=BF16, device="cuda")
    y[-3:] = torch.randn(3, n_out, generator=gen, device="cuda").bfloat16()
    tail = y[-3:].clone()
    idx, cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda"), torch.tensor([0, rows - 3, rows], dtype=torch.int32, device="cuda")
    cuda_lib.kda_lora(x, a, b, idx, y, cu_seqlens=cu, out=y)
    alone = cuda_lib.kda_lora(x[-3:].contiguous(), a, b, idx[1:], tail, cu_seqlens=torch.tensor([0, 3], dtype=torch.int32, device="cuda"))
    # the sums over 64 columns run in another order of parts: half a step of bf16
    assert off(y[-3:], alone.double().cpu().numpy()) <= 2.0 ** -8
    first = cuda_lib.kda_lora(x[:3].contiguous(), a, b, idx[:1], torch.zeros_like(tail), cu_seqlens=torch.tensor([0, 3], dtype=torch.int32, device="cuda"))
    assert off(y[:3], first.double().cpu().numpy()) <= 2.0 ** -8


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_many_requests(cuda_lib, dtype):
    """More requests than a warp looks at in one turn, empty ones among them, one adapter for several."""
    gen = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 4, (150,), generator=gen).tolist()
    run(cuda_lib, problem(lens, 192, 136, 8, adapters=7, dtype=dtype, seed=4))


def test_more_requests_than_a_block_lists(cuda_lib):
    run(cuda_lib, problem([1] * 2500, 64, 64, 4, adapters=300, seed=5))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_behind_the_last_request(cuda_lib, dtype):
    p = problem([30, 100], 128, 96, 8, dtype=dtype, tail=75, idx=[1, 0])
    out, (dx, da, db) = forward(cuda_lib, p), backward(cuda_lib, p)
    check(p, [out, dx, da, db], reference(p))
    assert torch.equal(out[130:].cpu(), p["y"][130:]) and torch.equal(dx[130:].cpu(), p["d_x"][130:])


def test_rows_without_adapter_keep_what_they_have(cuda_lib):
    p = problem([20, 70, 40], 128, 96, 8, idx=[-1, 1, 3])
    p["x"][:20] = float("nan")  # what is not used may hold anything
    p["x"][90:] = float("inf")
    out, (dx, da, db) = forward(cuda_lib, p), backward(cuda_lib, p)
    for r in (slice(0, 20), slice(90, 130)):
        assert torch.equal(out[r].cpu(), p["y"][r]) and torch.equal(dx[r].cpu(), p["d_x"][r])
    check(p, [out, dx, da, db], reference(p))
    assert float(da[[0, 2]].abs().max()) == 0 and float(db[[0, 2]].abs().max()) == 0


def test_in_place_and_partial_calls(cuda_lib):
    p = problem([64, 3], 256, 128, 16, idx=[0, 1])
    want, (dx, da, db) = forward(cuda_lib, p), backward(cuda_lib, p)
    d = cuda(p)
    got = cuda_lib.kda_lora(d["x"], d["a"], d["b"], d["idx"], d["y"], cu_seqlens=d["cu"], scale=d["scale"], out=d["y"])
    assert got is d["y"] and torch.equal(got, want)
    r = cuda_lib.kda_lora_bwd(d["d_out"], d["x"], d["a"], d["b"], d["idx"], d["d_x"], cu_seqlens=d["cu"], scale=d["scale"],
                              dx=d["d_x"], want_weights=False)
    assert r[0] is d["d_x"] and torch.equal(r[0], dx) and r[1] is None and r[2] is None
    r = backward(cuda_lib, p, want_dx=False)
    assert r[0] is None and torch.equal(r[1], da) and torch.equal(r[2], db)
    p["scale"] = torch.ones_like(p["scale"])
    d = cuda(p)
    plain = cuda_lib.kda_lora(d["x"], d["a"], d["b"], d["idx"], d["y"], cu_seqlens=d["cu"])
    assert torch.equal(plain, forward(cuda_lib, p))
    none = cuda_lib.kda_lora_bwd(d["d_out"], d["x"], d["a"], d["b"], d["idx"], cu_seqlens=d["cu"])[0]
    p["d_x"] = torch.zeros_like(p["d_x"])
    assert off(none, reference(p)[1]) <= TOL[BF16]


def test_the_same_each_time(cuda_lib):
    p = problem([1500, 900, 600], 512, 768, 32, adapters=2, idx=[0, 1, 0])
    one, two = [forward(cuda_lib, p), *backward(cuda_lib, p)], [forward(cuda_lib, p), *backward(cuda_lib, p)]
    assert all(torch.equal(a, b) for a, b in zip(one, two))
    check(p, one, reference(p))


def test_long_sums(cuda_lib):
    """All terms of one sign: the tensor core's cut-off sums would show."""
    p = problem([8192], 512, 256, 8, adapters=1, idx=[0], dtype=BF16)
    for n in ("x", "a", "b", "d_out"):
        p[n] = p[n].abs()
    check(p, [None, *backward(cuda_lib, p)], reference(p))


def test_no_rows(cuda_lib):
    p = problem([0, 0], 64, 32, 4, idx=[0, 1])
    assert forward(cuda_lib, p).shape == (0, 32)
    dx, da, db = backward(cuda_lib, p)
    assert dx.shape == (0, 64) and float(da.abs().max()) == 0 and float(db.abs().max()) == 0


def test_beside_the_8_bit_projection(cuda_lib):
    """As a server runs it: the norm to 8 bits, the shared projection, each request's adapter on the norm's bf16
    result; against the same in 64 bits on the values the 8-bit operands stand for."""
    import fp8_testutil
    kda = cuda_lib
    p = problem([40, 1, 90], 512, 384, 16, idx=[2, -1, 0])
    d = cuda(p)
    n = kda.kda_rms_norm(d["x"], fp8=True)
    w8, = kda.kda_fp8_quantize(torch.randn(384, 512, device="cuda") / 20, "tile")
    y = kda.kda_fp8_matmul(n.fp8, w8)
    got = kda.kda_lora(n.out, d["a"], d["b"], d["idx"], y, cu_seqlens=d["cu"], scale=d["scale"])
    p["x"], p["y"] = n.out.cpu(), torch.tensor(fp8_testutil.values(n.fp8) @ fp8_testutil.values(w8).T)
    # y is rounded to bf16 on the way: one more half step
    assert off(got, reference(p)[0]) <= 2 * 2.0 ** -8
