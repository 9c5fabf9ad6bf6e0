"""The gated delta rule and the adapters as they are used: a layer's projections with the requests' adapters, packed
prefill into a pool of states, decode on it, and the layer's gradients; the calls in captured graphs, on other streams
and from several threads."""
import threading

import numpy as np
import pytest
import torch

import fp8_testutil
import oracle
from gdn_testutil import EPS, TOL, args, cuda, off, oracle_of, problem
from test_lora import forward as lora_forward
from test_lora import backward as lora_backward
from test_lora import problem as lora_problem

pytestmark = pytest.mark.gpu

D, H, HK, DK, DV = 256, 4, 2, 64, 64
WIDTHS = dict(q=HK * DK, k=HK * DK, v=H * DV, g=H, beta=H)


class Layer:
    """Projections of one width D with adapters for each, then the gated delta rule; and the same in 64 bits."""

    def __init__(self, kda, adapters=3, rank=8, seed=0):
        gen = torch.Generator().manual_seed(seed)

        def randn(*s):
            return torch.randn(*s, generator=gen)
        self.kda = kda
        self.w = {n: (randn(w, D) * D ** -0.5) for n, w in WIDTHS.items()}
        self.w8 = {n: kda.kda_fp8_quantize(w.cuda(), "tile")[0] for n, w in self.w.items()}
        self.a = {n: (randn(adapters, rank, D) * D ** -0.5).bfloat16().cuda() for n in WIDTHS}
        self.b = {n: (0.2 * randn(adapters, w, rank)).bfloat16().cuda() for n, w in WIDTHS.items()}
        self.scale = torch.full((adapters,), 2.0, device="cuda")
        self.gate = dict(a_log=(-2 * torch.rand(H, generator=gen)).cuda(), dt_bias=randn(H).cuda(), gate_in_kernel=True,
                         beta_sigmoid=True, eps=EPS, scale=DK ** -0.5)

    def project(self, x, idx, cu):
        n = self.kda.kda_rms_norm(x, fp8=True)
        out = {}
        for name in WIDTHS:
            y = self.kda.kda_fp8_matmul(n.fp8, self.w8[name])
            y = self.kda.kda_lora(n.out, self.a[name], self.b[name], idx, y, cu_seqlens=cu, scale=self.scale, out=y)
            out[name] = y
        rows = x.shape[0]
        return (out["q"].view(rows, HK, DK), out["k"].view(rows, HK, DK), out["v"].view(rows, H, DV), out["g"].float(),
                out["beta"].float())

    def project64(self, x, idx, spans):
        """On the 8-bit values the library's norm and quantiser give (those have their own tests)."""
        n = self.kda.kda_rms_norm(x, fp8=True)
        n8, n16 = fp8_testutil.values(n.fp8), n.out.double().cpu().numpy()
        out = {}
        for name in WIDTHS:
            y = n8 @ fp8_testutil.values(self.w8[name]).T
            for (r0, r1), l in zip(spans, idx):
                if 0 <= l < self.scale.numel():
                    a, b = self.a[name][l].double().cpu().numpy(), self.b[name][l].double().cpu().numpy()
                    y[r0:r1] += 2.0 * (n16[r0:r1] @ a.T) @ b.T
            out[name] = y
        return out


def test_prefill_and_decode_of_requests_with_adapters(cuda_lib):
    """Against the 64-bit oracle fed with the projections that the library's calls gave (bf16), and these against 64 bits."""
    kda, layer = cuda_lib, Layer(cuda_lib)
    lens, adapters = [40, 1, 97, 64], [2, -1, 0, 2]
    cu = np.concatenate([[0], np.cumsum(lens)])
    gen = torch.Generator().manual_seed(1)
    steps = 3
    x = torch.randn(cu[-1], D, generator=gen).bfloat16().cuda()
    later = torch.randn(steps, len(lens), D, generator=gen).bfloat16().cuda()
    idx, rows = torch.tensor(adapters, dtype=torch.int32, device="cuda"), torch.tensor([5, 0, 3, 7], dtype=torch.int32, device="cuda")
    cu_dev = torch.tensor(cu, dtype=torch.int32, device="cuda")
    pool = torch.full((9, H, DK, DV), 3.0, device="cuda")

    p = layer.project(x, idx, cu_dev)
    want = layer.project64(x, adapters, [(cu[i], cu[i + 1]) for i in range(len(lens))])
    for name, got in zip(WIDTHS, p):
        # the 8-bit product and the adapter's sum are each rounded to bf16 once
        assert off(got.reshape(cu[-1], -1), want[name]) <= 2 * 2.0 ** -8, name
    out, state = kda.kda_gdn_chunk_fwd(*p, cu_seqlens=cu_dev, **layer.gate)
    kda.kda_state_scatter(pool, rows, state)
    tokens = [[t[cu[i]:cu[i + 1]] for t in p] for i in range(len(lens))]
    outs = [[out[cu[i]:cu[i + 1]]] for i in range(len(lens))]
    for t in range(steps):
        d = layer.project(later[t], idx, None)
        o = kda.kda_gdn_recurrent_step(*(y.unsqueeze(1) for y in d), pool, rows, **layer.gate)
        for i in range(len(lens)):
            tokens[i] = [torch.cat([a, b[i:i + 1]]) for a, b in zip(tokens[i], d)]
            outs[i].append(o[i])
    for i in range(len(lens)):
        T = lens[i] + steps
        q, k, v, g, beta = (y.double().cpu() for y in tokens[i])
        ref = oracle.Problem(q.repeat_interleave(H // HK, 1), k.repeat_interleave(H // HK, 1), v, g[..., None].expand(T, H, DK), beta,
                             cu_seqlens=[0, T], scale=layer.gate["scale"], eps=EPS, a_log=layer.gate["a_log"],
                             dt_bias=layer.gate["dt_bias"][:, None].expand(H, DK), beta_sigmoid=True, gate_in_kernel=True)
        o, f = oracle.chunk_fwd(ref)
        assert off(torch.cat(outs[i]), o) <= TOL[torch.bfloat16]
        assert off(pool[rows[i]], f[0]) <= TOL[torch.float32]
    assert bool((pool[[1, 2, 4, 6, 8]] == 3).all())


def test_gradients_of_a_layer_with_adapters(cuda_lib):
    """v's projection with its adapters and the rule after it, differentiated by the calls' own gradients put together,
    against differences of the 64-bit chain."""
    kda = cuda_lib
    p = problem([50, 31], hk=HK, h=H, dk=DK, dv=DV, dtype=torch.float32, seed=2)
    l = lora_problem([50, 31], D, H * DV, 4, adapters=2, dtype=torch.float32, idx=[1, 0], seed=3)
    d, e = cuda(p), cuda(l)
    v = kda.kda_lora(e["x"], e["a"], e["b"], e["idx"], e["y"], cu_seqlens=e["cu"], scale=e["scale"])
    g = kda.kda_gdn_chunk_bwd(d["q"], d["k"], v.view(81, H, DV), d["g"], d["beta"], d["d_out"], d_final_state=d["d_final"], **d["kw"])
    dx, da, db = kda.kda_lora_bwd(g["dv"].view(81, -1), e["x"], e["a"], e["b"], e["idx"], cu_seqlens=e["cu"], scale=e["scale"])

    def loss(x, a, b):
        y = l["y"].double().clone()
        for r0, r1, m in l["spans"]:
            y[r0:r1] += l["scale"][m].double() * (x[r0:r1] @ a[m].t()) @ b[m].t()
        o, f = oracle.chunk_fwd(oracle_of(dict(p, v=y.view(81, H, DV))), p["kw"]["initial_state"])
        return (o * p["d_out"].double().numpy()).sum() + (f * p["d_final"].double().numpy()).sum()
    at = {n: l[n].double() for n in "xab"}
    gen = torch.Generator().manual_seed(4)
    for n, got in (("x", dx), ("a", da), ("b", db)):
        u = torch.randn(at[n].shape, generator=gen, dtype=torch.float64)
        # the loss is linear in v and so in each of these: differences are exact but for 64-bit rounding
        slope = (loss(**{**at, n: at[n] + u}) - loss(**{**at, n: at[n] - u})) / 2
        mine = float((got.double().cpu() * u).sum())
        size = float(got.double().norm()) * float(u.norm()) / u.numel() ** 0.5
        assert abs(slope - mine) <= 2e-5 * (abs(slope) + size), n


def _calls(kda):
    """Each operator on its own inputs, as (name, call) with tensors to compare."""
    p, l = cuda(problem([200, 64, 3], hk=2, h=4, seed=1)), cuda(lora_problem([100, 33, 7], 256, 264, 16, idx=[1, 0, 2], seed=2))
    many = cuda(problem([580] * 10, hk=4, h=8, seed=5, packed=False))
    step = cuda(problem([1] * 5, packed=False, seed=3))
    kw = {n: v for n, v in step["kw"].items() if n not in ("initial_state", "cu_seqlens")}
    idx, pool = torch.tensor([3, 1, 0, 6, 2], device="cuda"), torch.randn(7, 4, 128, 128, device="cuda") / 10

    def decode():
        mine = pool.clone()
        return kda.kda_gdn_recurrent_step(*args(step), mine, idx, **kw), mine
    return [("fwd", lambda: kda.kda_gdn_chunk_fwd(*args(p), **p["kw"])),
            ("fwd, many heads", lambda: kda.kda_gdn_chunk_fwd(*args(many), **many["kw"])),
            ("bwd", lambda: tuple(kda.kda_gdn_chunk_bwd(*args(p), p["d_out"], d_final_state=p["d_final"], **p["kw"]).values())),
            ("step", decode),
            ("lora", lambda: (kda.kda_lora(l["x"], l["a"], l["b"], l["idx"], l["y"], cu_seqlens=l["cu"], scale=l["scale"]),)),
            ("lora bwd", lambda: kda.kda_lora_bwd(l["d_out"], l["x"], l["a"], l["b"], l["idx"], l["d_x"], cu_seqlens=l["cu"],
                                                  scale=l["scale"]))]


def _same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_captured_and_replayed(cuda_lib):
    for name, call in _calls(cuda_lib):
        want = call()
        g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(g, stream=s):
            got = call()
        for t in got:
            t.zero_()
        for _ in range(2):
            g.replay()
        torch.cuda.synchronize()
        assert _same(got, want), name


def test_all_at_once_on_several_streams(cuda_lib):
    calls = _calls(cuda_lib)
    wants = [call() for _, call in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2 * len(calls))]
    gots = []
    for i, s in enumerate(streams):
        with torch.cuda.stream(s):
            gots.append([calls[i % len(calls)][1]() for _ in range(5)])
    torch.cuda.synchronize()
    for i, got in enumerate(gots):
        for g in got:
            assert _same(g, wants[i % len(calls)]), calls[i % len(calls)][0]


def test_from_several_threads(cuda_lib):
    calls = _calls(cuda_lib)
    wants = [call() for _, call in calls]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(10):
                    got = calls[i][1]()
                    s.synchronize()
                    if not _same(got, wants[i]):
                        bad.append(calls[i][0])
        except Exception as e:  # noqa: B902
            bad.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_given_streams(cuda_lib):
    kda = cuda_lib
    p, l = problem([90, 40], seed=1), lora_problem([90, 40], 128, 64, 8, idx=[0, 1])
    d = cuda(p)
    want = kda.kda_gdn_chunk_fwd(*args(d), **d["kw"])
    want_b = kda.kda_gdn_chunk_bwd(*args(d), d["d_out"], **d["kw"])
    want_l, want_lb = lora_forward(kda, l), lora_backward(kda, l)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = kda.kda_gdn_chunk_fwd(*args(d), stream=s, **d["kw"])
    got_b = kda.kda_gdn_chunk_bwd(*args(d), d["d_out"], stream=s, **d["kw"])
    s.synchronize()
    assert _same(got, want) and all(torch.equal(got_b[n], want_b[n]) for n in want_b if want_b[n] is not None)
    e = cuda(l)
    torch.cuda.synchronize()
    got_l = kda.kda_lora(e["x"], e["a"], e["b"], e["idx"], e["y"], cu_seqlens=e["cu"], scale=e["scale"], stream=s)
    got_lb = kda.kda_lora_bwd(e["d_out"], e["x"], e["a"], e["b"], e["idx"], e["d_x"], cu_seqlens=e["cu"], scale=e["scale"], stream=s)
    s.synchronize()
    assert torch.equal(got_l, want_l) and _same(got_lb, want_lb)
