"""The gated delta rule with one gate per head (chunked forward and backward, recurrent step on pool states)
and low-rank adapters of many requests beside a shared projection (forward and backward), as cases to measure.

Gated delta rule, per value head (the key heads of q and k are shared by groups of value heads):
    S_t = exp(g_t) (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T,   o_t = scale S_t^T q_t
with k, q after their L2 norm, beta the sigmoid of a logit, g = -exp(a_log) softplus(x + dt_bias) <= 0.

Adapters: the rows of request i take adapter l = idx[i] (none if l is out of range):
    out = y + scale[l] (x A[l]^T) B[l]^T,   A [adapters, rank, n_in], B [adapters, n_out, rank]

Cases are dicts: "op" is gdn, gdn_bwd, step, lora or lora_bwd; the other keys are its sizes and options.
"""
import math

import torch

own = False

EPS = 1e-6
CHUNK = 64
# a drawn case costs no more than the largest listed ones: value-head tokens, states of a step, elements of x and y
MOST_TOKEN_HEADS = 4 * 8192 * 32
MOST_STATES = 64 * 32
MOST_ELEMS = 32768 * 8192


def listed():
    return [
        # the end of one short prompt after a cached prefix: two heads, 130 tokens; latency
        dict(name="gdn_short", op="gdn", lens="1x130", hk=2, h=2, dk=128, dv=128, dtype="bf16", gate="slow"),
        # prefill of 16 packed requests, among them an empty one and one of a single token; grouped key heads
        dict(name="gdn_packed", op="gdn", lens="0,1,64,65,127,200,333,512,700,801,64,999,1024,1030,1100,1171", hk=8, h=16, dk=128, dv=128, dtype="bf16", gate="slow"),
        # fp32 tensors, heads of 64, a length that is no multiple of the chunk, gates that decay by several nats a token
        dict(name="gdn_f32", op="gdn", lens="2x1001", hk=4, h=8, dk=64, dv=64, dtype="f32", gate="strong"),
        # the training batch of 4 x 8192 tokens, 32 value heads on 16 key heads
        dict(name="gdn_train", op="gdn", lens="4x8192", hk=16, h=32, dk=128, dv=128, dtype="bf16", gate="slow"),
        # its gradients on a few short documents packed together, narrow value heads
        dict(name="gdn_bwd_packed", op="gdn_bwd", lens="5,300,0,64,257,130", hk=2, h=4, dk=128, dv=64, dtype="bf16", gate="slow"),
        # the training batch's gradients
        dict(name="gdn_bwd_train", op="gdn_bwd", lens="4x8192", hk=16, h=32, dk=128, dv=128, dtype="bf16", gate="slow"),
        # one token of one sequence, 32 heads: latency of the recurrent step
        dict(name="step_one", op="step", n=1, t=1, hk=16, h=32, dk=128, dv=128, dtype="bf16", cache="f32"),
        # a decode batch of 64 sequences: the states' bytes
        dict(name="step_batch", op="step", n=64, t=1, hk=16, h=32, dk=128, dv=128, dtype="bf16", cache="f32"),
        # a decode batch of 64 requests, each with one of 48 adapters, a few without
        dict(name="lora_decode", op="lora", lens="64x1", n_in=4096, n_out=4096, rank=16, adapters=48, dtype="bf16"),
        # prefill of 9 packed requests of odd lengths on 5 adapters, widths of 16 heads x 128 and 4196
        dict(name="lora_packed", op="lora", lens="1,777,1500,0,31,2048,64,999,1311", n_in=2048, n_out=4196, rank=24, adapters=5, dtype="bf16"),
        # fine-tuning two adapters on short documents: all gradients
        dict(name="lora_bwd_packed", op="lora_bwd", lens="130,64,1,301", n_in=1024, n_out=2048, rank=8, adapters=2, dtype="bf16"),
        # the training batch of 4 x 8192 tokens on 4 adapters, width 32 heads x 128: all gradients
        dict(name="lora_bwd_train", op="lora_bwd", lens="4x8192", n_in=4096, n_out=4096, rank=64, adapters=4, dtype="bf16"),
    ]


def _lens(case):
    s = case["lens"]
    if "x" in s:
        n, t = s.split("x")
        return [int(t)] * int(n)
    return [int(t) for t in s.split(",")]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_lens(rng, most):
    """Equal sequences, or packed ones of any lengths, up to `most` tokens in all."""
    most = max(1, min(most, 32768))
    if rng.random() < 0.4:
        n = min(rng.choice([1, 2, 4, 7]), most)
        return "%dx%d" % (n, _log_uniform(rng, 1, min(8192, most // n)))
    total, lens = _log_uniform(rng, 1, most), []
    while total > 0 and len(lens) < 40:
        t = min(total, rng.choice([0, 1, 63, _log_uniform(rng, 1, 8192), _log_uniform(rng, 1, 8192), _log_uniform(rng, 1, 8192)]))
        lens.append(t)
        total -= t
    return ",".join(map(str, lens + [0] * (len(lens) < 2)))


def draw(rng):
    op = rng.choice(["gdn", "gdn", "gdn_bwd", "gdn_bwd", "step", "lora", "lora", "lora_bwd"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op in ("gdn", "gdn_bwd", "step"):
        hk = rng.choice([1, 2, 3, 4, 8, 16])
        h = hk * rng.choice([1, 1, 2, 2, 3, 4])
        c = dict(op=op, hk=hk, h=min(h, 32 // hk * hk), dk=rng.choice([64, 128, 128]), dv=rng.choice([64, 128, 128]), dtype=dtype)
        if op == "step":
            t = rng.choice([1, 1, 1, 2, 3, 5])
            return dict(c, n=_log_uniform(rng, 1, max(1, MOST_STATES // (c["h"] * t))), t=t, cache=rng.choice(["f32", "f32", "bf16"]))
        most = MOST_TOKEN_HEADS // c["h"] // (4 if dtype == "f32" else 1)
        return dict(c, lens=_draw_lens(rng, most), gate=rng.choice(["slow", "slow", "strong"]))
    n_in, n_out = (w * 8 if rng.random() < 0.7 else w * 8 - rng.randrange(8) for w in (_log_uniform(rng, 8, 1024) for _ in range(2)))
    rank, adapters = rng.choice([1, 4, 8, 8, 13, 16, 16, 32, 64, 100, 128]), rng.choice([1, 2, 5, 16, 40])
    most = MOST_ELEMS // (n_in + n_out) // (8 if dtype == "f32" else 1) * 64 // max(64, rank)
    lens = "%dx1" % _log_uniform(rng, 1, 256) if rng.random() < 0.4 else _draw_lens(rng, most)
    return dict(op=op, lens=lens, n_in=n_in, n_out=n_out, rank=rank, adapters=adapters, dtype=dtype)


# ---------------------------------------------------------------- inputs

def _dtype(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _offsets(lens):
    cu = [0]
    for t in lens:
        cu.append(cu[-1] + t)
    return cu


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) % (1 << 62))

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    def rand(*shape):
        return torch.rand(*shape, device="cuda", generator=gen)

    if case["op"].startswith("lora"):
        return _prepare_lora(case, randn, rand)
    dtype = _dtype(case["dtype"])
    hk, h, dk, dv = case["hk"], case["h"], case["dk"], case["dv"]
    s = dict(case=case, scale=dk ** -0.5)
    if case["op"] == "step":
        n, t = case["n"], case["t"]
        lead = (n, t)
        rows = n + n // 2 + 1
        s["cache"] = (0.1 * randn(rows, h, dk, dv)).to(_dtype(case["cache"]))
        idx = torch.randperm(rows, device="cuda", generator=gen)[:n].to(torch.int32)
        flags = torch.ones(n, dtype=torch.bool, device="cuda")
        if n > 8:  # a padded slot of the batch, and a sequence that starts here
            idx[3] = -1
            flags[5] = False
        s["idx"], s["flags"] = idx, flags
    else:
        lens = _lens(case)
        s["lens"] = lens
        packed = "," in case["lens"]
        lead = (sum(lens),) if packed else (len(lens), lens[0])
        s["cu"] = torch.tensor(_offsets(lens), dtype=torch.int32, device="cuda") if packed else None
        s["initial"] = 0.1 * randn(len(lens), h, dk, dv)
    for name, heads, d in (("q", hk, dk), ("k", hk, dk), ("v", h, dv)):
        s[name] = randn(*lead, heads, d).to(dtype)
    s["g"], s["beta"] = randn(*lead, h), randn(*lead, h)
    lo, hi = (1.0, 3.0) if case.get("gate") == "strong" else (-4.0, 0.0)
    s["a_log"], s["dt_bias"] = lo + (hi - lo) * rand(h), 0.1 * randn(h)
    if case["op"] == "gdn_bwd":
        s["d_out"] = randn(*lead, h, dv).to(dtype)
        s["d_final"] = 0.1 * randn(len(lens), h, dk, dv)
    return s


def _prepare_lora(case, randn, rand):
    dtype, lens = _dtype(case["dtype"]), _lens(case)
    rows, n_in, n_out, r, many = sum(lens), case["n_in"], case["n_out"], case["rank"], case["adapters"]
    x = randn(rows, n_in) * torch.exp(0.5 * randn(rows, 1)) * (1 + 15 * (rand(1, n_in) < 0.005))
    s = dict(case=case, lens=lens, x=x.to(dtype), a=(randn(many, r, n_in) * n_in ** -0.5).to(dtype),
             b=(0.05 * randn(many, n_out, r)).to(dtype), scale=16.0 / r * (0.5 + rand(many)))
    # every row is a request of its own in decode; else the requests' rows follow one another
    s["cu"] = None if all(t == 1 for t in lens) else torch.tensor(_offsets(lens), dtype=torch.int32, device="cuda")
    s["idx"] = (rand(len(lens)) * many).to(torch.int32)
    if len(lens) > 6:  # requests without an adapter
        s["idx"][5::16] = -1
    if case["op"] == "lora":
        s["y"] = randn(rows, n_out).to(dtype)
    else:
        s["d_out"], s["d_x"] = (0.1 * randn(rows, n_out)).to(dtype), (0.1 * randn(rows, n_in)).to(dtype)
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import chunked_kimi_delta_gb300 as kda
    op = s["case"]["op"]
    if op == "lora":
        return kda.kda_lora(s["x"], s["a"], s["b"], s["idx"], s["y"], cu_seqlens=s["cu"], scale=s["scale"])
    if op == "lora_bwd":
        return list(kda.kda_lora_bwd(s["d_out"], s["x"], s["a"], s["b"], s["idx"], s["d_x"], cu_seqlens=s["cu"], scale=s["scale"]))
    kw = dict(scale=s["scale"], eps=EPS, a_log=s["a_log"], dt_bias=s["dt_bias"], beta_sigmoid=True, gate_in_kernel=True)
    args = (s["q"], s["k"], s["v"], s["g"], s["beta"])
    if op == "step":
        out = kda.kda_gdn_recurrent_step(*args, s["cache"], s["idx"], s["flags"], **kw)
        return [out, s["cache"]]
    kw.update(initial_state=s["initial"], cu_seqlens=s["cu"])
    if op == "gdn":
        return list(kda.kda_gdn_chunk_fwd(*args, **kw))
    d = kda.kda_gdn_chunk_bwd(*args, s["d_out"], d_final_state=s["d_final"], **kw)
    return [d[n] for n in ("dq", "dk", "dv", "dg", "dbeta", "da_log", "ddt_bias", "d_initial_state")]


def _run_plain(s):
    op = s["case"]["op"]
    if op.startswith("lora"):
        return _plain_lora(s) if op == "lora" else _plain_lora_bwd(s)
    if op == "step":
        return _plain_step(s)
    return _plain_chunked(s, op == "gdn_bwd")


def _activated(s, dt):
    """q, k after their norm and 1 / norm, log-decay, beta, from what the caller gives."""
    def normed(x):
        r = torch.rsqrt(x.square().sum(-1, keepdim=True) + EPS)
        return x * r, r
    q, rq = normed(s["q"].to(dt))
    k, rk = normed(s["k"].to(dt))
    z = s["g"].double() + s["dt_bias"].double()
    g = -torch.exp(s["a_log"].double()) * (z.clamp(min=0) + torch.log1p(torch.exp(-z.abs())))
    return q, rq, k, rk, g, torch.sigmoid(s["beta"].to(dt)), z


def _to_chunks(x, lens, tmax):
    """[tokens, heads, d] of sequences that follow one another -> [sequences, heads, chunks, CHUNK, d], zeros behind each."""
    out = x.new_zeros(len(lens), tmax, *x.shape[1:])
    at = torch.cat([torch.arange(t, device=x.device) + n * tmax for n, t in enumerate(lens)]) if len(set(lens)) > 1 else None
    if at is None:
        out[:, :lens[0]] = x.view(len(lens), lens[0], *x.shape[1:])
    else:
        out.view(len(lens) * tmax, *x.shape[1:])[at] = x
    return out.view(len(lens), tmax // CHUNK, CHUNK, *x.shape[1:]).permute(0, 3, 1, 2, 4).contiguous(), at


def _from_chunks(x, lens, at):
    n, h, c, t, d = x.shape
    x = x.permute(0, 2, 3, 1, 4).reshape(n, c * t, h, d)
    return x[:, :lens[0]].reshape(-1, h, d) if at is None else x.reshape(n * c * t, h, d)[at]


def _unit_lower_inverse(low):
    """(I + low)^-1 of strictly lower triangular matrices, row by row."""
    a = torch.zeros_like(low)
    for i in range(low.shape[-1]):
        a[..., i, :] = -torch.matmul(low[..., i:i + 1, :i], a[..., :i, :]).squeeze(-2)
        a[..., i, i] += 1
    return a


def _plain_chunked(s, backward):
    """The chunked form: inside a chunk (I + L) V' = beta (v - e^G k S), between chunks the state alone."""
    lens, scale = s["lens"], s["scale"]
    heads, group = s["case"]["h"], s["case"]["h"] // s["case"]["hk"]
    tmax = max(1, -(-max(lens) // CHUNK)) * CHUNK
    shape = s["v"].shape[:-2]
    q, rq, k, rk, g, beta, z = _activated(s, torch.float32)

    def chunks(x):
        return _to_chunks(x.reshape(-1, *x.shape[len(shape):]), lens, tmax)

    (Q, at), K, V = chunks(q), chunks(k)[0], chunks(s["v"].float())[0]
    Q, K = (x.repeat_interleave(group, 1) for x in (Q, K))
    b, G = chunks(beta[..., None])[0], chunks(g[..., None])[0].cumsum(-2)
    ones = torch.ones(CHUNK, CHUNK, device=q.device)
    diff = G - G.transpose(-1, -2)
    gamma = torch.where(ones.tril() > 0, torch.exp(diff.clamp(max=0)), 0.0).float()
    e, f, ec = torch.exp(G).float(), torch.exp(G[..., -1:, :] - G).float(), torch.exp(G[..., -1:, :]).float()
    KK = gamma * torch.matmul(K, K.transpose(-1, -2)) * (ones.tril(-1) > 0)
    A = _unit_lower_inverse(b * KK)
    P = gamma * torch.matmul(Q, K.transpose(-1, -2))
    S = s["initial"].float()
    n_chunks = Q.shape[2]
    O, kept = torch.empty_like(V), []
    for c in range(n_chunks):  # from chunk to chunk
        R = V[:, :, c] - e[:, :, c] * torch.matmul(K[:, :, c], S)
        W = torch.matmul(A[:, :, c], b[:, :, c] * R)
        if backward:
            kept.append((S, R, W))
        O[:, :, c] = scale * (e[:, :, c] * torch.matmul(Q[:, :, c], S) + torch.matmul(P[:, :, c], W))
        S = ec[:, :, c] * S + torch.matmul((f[:, :, c] * K[:, :, c]).transpose(-1, -2), W)
    if not backward:
        return [_from_chunks(O, lens, at).view(s["v"].shape).to(s["v"].dtype), S]

    D = scale * chunks(s["d_out"].float())[0]
    dQ, dK, dV, dG, db = torch.empty_like(Q), torch.empty_like(K), torch.empty_like(V), torch.zeros_like(e), torch.empty_like(b)
    dS = s["d_final"].float()
    for c in reversed(range(n_chunks)):
        S, R, W = kept.pop()
        k_, q_, d_, b_, e_, f_, ec_ = (x[:, :, c] for x in (K, Q, D, b, e, f, ec))
        kdS = torch.matmul(k_, dS)
        dW = torch.matmul(P[:, :, c].transpose(-1, -2), d_) + f_ * kdS
        dY = torch.matmul(A[:, :, c].transpose(-1, -2), dW)
        dR = b_ * dY
        dP = torch.matmul(d_, W.transpose(-1, -2)) * gamma[:, :, c]
        dL = -torch.matmul(dY, W.transpose(-1, -2)) * gamma[:, :, c] * (ones.tril(-1) > 0)
        inside = dL * torch.matmul(k_, k_.transpose(-1, -2))
        db[:, :, c] = (dY * R).sum(-1, keepdim=True) + inside.sum(-1, keepdim=True)
        X = dP * torch.matmul(q_, k_.transpose(-1, -2)) + b_ * inside
        qS, kS = torch.matmul(d_, S.transpose(-1, -2)), torch.matmul(dR, S.transpose(-1, -2))
        WdS = torch.matmul(W, dS.transpose(-1, -2))
        y = f_ * (W * kdS).sum(-1, keepdim=True)
        # the gate at r scales what crosses it: pairs i >= r > j, the state's way to i >= r, that of j < r to the next state, and the state's own
        across = (X.flip(-2).cumsum(-2).flip(-2) * ones.tril(-1)).sum(-1, keepdim=True)
        inter = e_ * ((qS * q_).sum(-1, keepdim=True) - (kS * k_).sum(-1, keepdim=True))
        dG[:, :, c] = across + inter.flip(-2).cumsum(-2).flip(-2) + torch.matmul(ones.tril(-1), y) + ec_ * (S * dS).sum((-1, -2)).unsqueeze(-1).unsqueeze(-1)
        M = b_ * dL
        dQ[:, :, c] = e_ * qS + torch.matmul(dP, k_)
        dK[:, :, c] = -e_ * kS + f_ * WdS + torch.matmul(dP.transpose(-1, -2), q_) + torch.matmul(M + M.transpose(-1, -2), k_)
        dV[:, :, c] = dR
        dS = ec_ * dS + torch.matmul((e_ * q_).transpose(-1, -2), d_) - torch.matmul((e_ * k_).transpose(-1, -2), dR)

    def back(x):
        return _from_chunks(x, lens, at).view(*shape, heads, -1)

    def unnormed(dx, x, r):
        dx = dx.view(*shape, heads // group, group, -1).sum(-2)
        return (r * (dx - x * (x * dx).sum(-1, keepdim=True)))
    dg, db = back(dG).squeeze(-1).double(), back(db).squeeze(-1)
    dx = -torch.exp(s["a_log"].double()) * torch.sigmoid(z) * dg
    over = tuple(range(len(shape)))
    t = s["v"].dtype
    return [unnormed(back(dQ), q, rq).to(t), unnormed(back(dK), k, rk).to(t), back(dV).to(t), dx.float(),
            db * beta * (1 - beta), (g * dg).sum(over).float(), dx.sum(over).float(), dS]


def _plain_step(s):
    q, _, k, _, g, beta, _ = _activated(s, torch.float32)
    group = s["case"]["h"] // s["case"]["hk"]
    q, k, v, a = q.repeat_interleave(group, 2), k.repeat_interleave(group, 2), s["v"].float(), torch.exp(g).float()
    cache, idx = s["cache"], s["idx"].long()
    valid = (idx >= 0) & (idx < cache.shape[0])
    S = torch.where((valid & s["flags"])[:, None, None, None], cache[idx.clamp(min=0)].float(), 0.0)
    out = torch.empty_like(v)
    for t in range(s["case"]["t"]):
        S = a[:, t, :, None, None] * S
        delta = beta[:, t, :, None] * (v[:, t] - (S * k[:, t, :, :, None]).sum(-2))
        S = S + k[:, t, :, :, None] * delta[:, :, None]
        out[:, t] = s["scale"] * (S * q[:, t, :, :, None]).sum(-2)
    cache[idx[valid]] = S[valid].to(cache.dtype)
    return [out.to(s["v"].dtype), cache]


def _requests(s):
    """(first row, end, adapter) of the requests that have one; the indices are read as whole numbers."""
    cu = _offsets(s["lens"])
    return [(cu[i], cu[i + 1], l) for i, l in enumerate(s["idx"].tolist()) if 0 <= l < s["a"].shape[0] and cu[i + 1] > cu[i]]


def _of_rows(s):
    """Each row's adapter (0 where it has none) and its factor (0 there)."""
    many = s["a"].shape[0]
    idx = s["idx"].long()
    fine = (idx >= 0) & (idx < many)
    idx = torch.where(fine, idx, torch.zeros_like(idx))
    f = torch.where(fine, s["scale"][idx], torch.zeros_like(s["scale"][idx]))
    if s["cu"] is not None:
        at = torch.searchsorted(s["cu"][1:].long(), torch.arange(s["x"].shape[0], device=f.device), right=True)
        idx, f = idx[at], f[at]
    return idx, f[:, None]


def _plain_lora(s):
    idx, f = _of_rows(s)
    x, out = s["x"].float(), s["y"].float()
    if s["cu"] is None:  # one row a request: its own adapter's matrices
        u = torch.matmul(s["a"].float()[idx], x[:, :, None])
        return (out + f * torch.matmul(s["b"].float()[idx], u).squeeze(-1)).to(s["y"].dtype)
    for l in range(s["a"].shape[0]):
        mine = f * (idx == l)[:, None]
        out = out + mine * torch.matmul(torch.matmul(x, s["a"][l].float().t()), s["b"][l].float().t())
    return out.to(s["y"].dtype)


def _plain_lora_bwd(s):
    idx, f = _of_rows(s)
    x, d, dx = s["x"].float(), s["d_out"].float(), s["d_x"].float()
    da, db = torch.empty_like(s["a"], dtype=torch.float32), torch.empty_like(s["b"], dtype=torch.float32)
    for l in range(s["a"].shape[0]):
        a, b, mine = s["a"][l].float(), s["b"][l].float(), f * (idx == l)[:, None]
        du = mine * torch.matmul(d, b)
        dx = dx + torch.matmul(du, a)
        da[l] = torch.matmul(du.t(), x)
        db[l] = torch.matmul(d.t(), mine * torch.matmul(x, a.t()))
    return [dx.to(s["x"].dtype), da, db]


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("lora"):
        lens = _lens(case)
        rows, r, wide = sum(lens), case["rank"], case["n_in"] + case["n_out"]
        used = min(case["adapters"], sum(t > 0 for t in lens))
        if case["op"] == "lora":  # x, y and the result; the matrices of the adapters in use
            return dict(bytes=e * (rows * (wide + case["n_out"]) + used * r * wide), flops=2.0 * rows * r * wide)
        return dict(bytes=e * (rows * (wide + 2 * case["n_in"]) + used * r * wide) + 4 * case["adapters"] * r * wide, flops=6.0 * rows * r * wide)
    hk, h, dk, dv = case["hk"], case["h"], case["dk"], case["dv"]
    if case["op"] == "step":
        tokens = case["n"] * case["t"]
        state = dk * dv * (2 if case["cache"] == "bf16" else 4)
        return dict(bytes=case["n"] * h * 2 * state + tokens * (e * (2 * hk * dk + 2 * h * dv) + 8 * h), flops=6.0 * tokens * h * dk * dv)
    lens = _lens(case)
    tokens, states = sum(lens), 4 * len(lens) * h * dk * dv
    # per value-head token, triangles once: the products of q k^T and k k^T, the solve, the three with the state, o's inner part
    flops = tokens * h * (6.0 * dk * dv + CHUNK * (2 * dk + 2 * dv))
    if case["op"] == "gdn":
        return dict(bytes=tokens * (e * (2 * hk * dk + 2 * h * dv) + 8 * h) + 2 * states, flops=flops)
    return dict(bytes=tokens * (e * (4 * hk * dk + 3 * h * dv) + 16 * h) + 3 * states, flops=tokens * h * (16.0 * dk * dv + CHUNK * (6 * dk + 6 * dv)))


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("lora"):
        return _exact_lora(s, case["op"] == "lora_bwd")
    for name in ("q", "k", "v", "g", "beta", "a_log", "dt_bias"):
        s[name] = s[name].double()
    if case["op"] == "step":
        return _exact_step(s)
    return _exact_recurrence(s, case["op"] == "gdn_bwd")


def _gate(s):
    return -torch.exp(s["a_log"]) * torch.logaddexp(s["g"] + s["dt_bias"], torch.zeros_like(s["g"]))


def _unit(x):
    return x / torch.sqrt((x * x).sum(-1, keepdim=True) + EPS)


def _exact_step(s):
    cache = s["cache"].double()
    hk, group, scale = s["case"]["hk"], s["case"]["h"] // s["case"]["hk"], s["scale"]
    out = torch.empty_like(s["v"])
    alpha, beta, q, k = torch.exp(_gate(s)), 1 / (1 + torch.exp(-s["beta"])), _unit(s["q"]), _unit(s["k"])
    for n, (row, flag) in enumerate(zip(s["idx"].tolist(), s["flags"].tolist())):
        valid = 0 <= row < cache.shape[0]
        S = cache[row] if valid and flag else torch.zeros_like(cache[0])
        for t in range(s["case"]["t"]):
            kk, qq = (x[n, t][:, None].expand(hk, group, -1).flatten(0, 1) for x in (k, q))
            S = alpha[n, t][:, None, None] * S
            got = torch.einsum("hkv,hk->hv", S, kk)
            S = S + torch.einsum("hk,hv->hkv", kk, beta[n, t][:, None] * (s["v"][n, t] - got))
            out[n, t] = scale * torch.einsum("hkv,hk->hv", S, qq)
        if valid:
            cache[row] = S
    return [out, cache]


class _Tokens:
    """The recurrence on all sequences at once, token by token, on rows ordered [step, sequence]; sequences that have
    ended keep their state (decay 1, beta 0, zero keys)."""

    def __init__(self, s):
        lens, h, hk = s["lens"], s["case"]["h"], s["case"]["hk"]
        n, steps = len(lens), max(lens)
        cu = torch.tensor(_offsets(lens), device="cuda")
        at = cu[:-1][None, :] + torch.arange(steps, device="cuda")[:, None]
        self.live = at < cu[1:][None, :]
        self.at = torch.where(self.live, at, torch.zeros_like(at))

        def rows(x):
            x = x.reshape(-1, *x.shape[len(s["v"].shape) - 2:])
            x = torch.where(self.live.view(steps, n, *([1] * (x.dim() - 1))), x[self.at], torch.zeros_like(x[:1]))
            return x.repeat_interleave(h // hk, 2) if x.dim() == 4 and x.shape[2] == hk and hk != h else x
        self.rows, self.steps = rows, steps
        self.q, self.k, self.v = rows(_unit(s["q"])), rows(_unit(s["k"])), rows(s["v"])
        self.alpha, self.beta = torch.exp(rows(_gate(s))), rows(torch.sigmoid(s["beta"]))

    def step(self, t, S):
        """The state before the decay's use is S; returns the error v - S'^T k and the new state."""
        S = S * self.alpha[t, :, :, None, None]
        err = self.v[t] - torch.matmul(self.k[t].unsqueeze(-2), S).squeeze(-2)
        return err, torch.addcmul(S, self.k[t].unsqueeze(-1), (self.beta[t][..., None] * err).unsqueeze(-2))


def _exact_recurrence(s, backward):
    lens, heads = s["lens"], s["case"]["h"]
    if max(lens) * len(lens) * heads * s["case"]["dk"] * s["case"]["dv"] * (4 if backward else 1) > 4e10:
        return None
    shape, scale = s["v"].shape[:-2], s["scale"]
    if max(lens) == 0:
        return None
    T = _Tokens(s)
    tokens = sum(lens)

    def back(x):
        """[step, sequence, ...] -> the caller's token order."""
        out = x.new_zeros(tokens, *x.shape[2:])
        out[T.at[T.live]] = x[T.live]
        return out.view(*shape, *x.shape[2:])

    S, every, kept = s["initial"].double(), 64, []
    O = torch.empty_like(T.v)
    for t in range(T.steps):
        if t % every == 0:
            kept.append(S)
        _, S = T.step(t, S)
        O[t] = scale * torch.matmul(T.q[t].unsqueeze(-2), S).squeeze(-2)
    if not backward:
        return [back(O), S]

    d_out, D = T.rows(s["d_out"].double()), s["d_final"].double()
    dq, dk, dv = torch.empty_like(T.q), torch.empty_like(T.k), torch.empty_like(T.v)
    dalpha, dbeta = torch.empty_like(T.alpha), torch.empty_like(T.beta)
    for start in reversed(range(0, T.steps, every)):
        S, states = kept.pop(), []
        for t in range(start, min(start + every, T.steps)):
            states.append(S)
            _, S = T.step(t, S)
        for t in reversed(range(start, start + len(states))):
            before = states.pop()
            err, after = T.step(t, before)
            g = scale * d_out[t]
            D = torch.addcmul(D, T.q[t].unsqueeze(-1), g.unsqueeze(-2))
            dq[t] = torch.matmul(after, g.unsqueeze(-1)).squeeze(-1)
            b = T.beta[t][..., None]
            Dk = torch.matmul(T.k[t].unsqueeze(-2), D).squeeze(-2)  # the new state is S' + k (b err)^T, err = v - S'^T k
            dbeta[t] = (Dk * err).sum(-1)
            dv[t] = b * Dk
            decayed = before * T.alpha[t, :, :, None, None]
            dk[t] = torch.matmul(D, (b * err).unsqueeze(-1)).squeeze(-1) - torch.matmul(decayed, dv[t].unsqueeze(-1)).squeeze(-1)
            D = torch.addcmul(D, T.k[t].unsqueeze(-1), dv[t].unsqueeze(-2), value=-1)
            dalpha[t] = (D * before).sum((-1, -2))
            D = D * T.alpha[t, :, :, None, None]
    hk = s["case"]["hk"]

    def through_norm(d, x):
        d = back(d).view(*shape, hk, heads // hk, -1).sum(-2)
        n2 = (x * x).sum(-1, keepdim=True) + EPS
        return d / n2.sqrt() - x * (x * d).sum(-1, keepdim=True) / n2 ** 1.5
    dlog = back(dalpha * T.alpha)
    beta = torch.sigmoid(s["beta"])
    dx = -torch.exp(s["a_log"]) * torch.sigmoid(s["g"] + s["dt_bias"]) * dlog
    over = tuple(range(len(shape)))
    return [through_norm(dq, s["q"]), through_norm(dk, s["k"]), back(dv), dx, back(dbeta) * beta * (1 - beta),
            (_gate(s) * dlog).sum(over), dx.sum(over), D]


def _exact_lora(s, backward):
    x, a, b, scale = (s[n].double() for n in ("x", "a", "b", "scale"))
    if not backward:
        out = s["y"].double()
        for first, end, l in _requests(s):
            out[first:end] += torch.einsum("tr,or->to", torch.einsum("ti,ri->tr", x[first:end], a[l]), scale[l] * b[l])
        return out
    d, dx = s["d_out"].double(), s["d_x"].double()
    da, db = torch.zeros_like(a), torch.zeros_like(b)
    for first, end, l in _requests(s):
        u, du = x[first:end] @ a[l].t(), scale[l] * (d[first:end] @ b[l])
        dx[first:end] += du @ a[l]
        da[l] += du.t() @ x[first:end]
        db[l] += scale[l] * (d[first:end].t() @ u)
    return [dx, da, db]
