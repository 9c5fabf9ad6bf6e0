"""Host-side checks of the gated delta rule with one gate per head and of the low-rank adapters, without a GPU: refusals
of the C calls and of the Python binding."""
import ctypes

import pytest
import torch

import chunked_kimi_delta_gb300 as kda
from chunked_kimi_delta_gb300 import build as kbuild

BASE = 1 << 20
INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 1, 2, 3, 4
LARGE = 1 << 40


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda.load_library()


def _fill(args, fields, /, **kw):
    for key, val in {**fields, **kw}.items():
        setattr(args, key, val)
    return args


FWD = dict(B=2, T=100, H=4, dk=128, dv=128, chunk=64, qkv_dtype=kda.KDA_BF16, q=BASE, k=2 * BASE, v=3 * BASE, g=4 * BASE,
           beta=5 * BASE, a_log=6 * BASE, scale=0.1, eps=1e-6, out=7 * BASE, final_state=8 * BASE, workspace=16 * BASE,
           workspace_bytes=LARGE, Hk=2, flags=kda.KDA_GATE_IN_KERNEL)


def _fwd(**kw):
    return _fill(kda.kda_fwd_args(), FWD, **kw)


def _bwd(fwd=None, **kw):
    b = _fill(kda.kda_bwd_args(), dict(d_out=BASE, d_final_state=2 * BASE, dq=3 * BASE, dk=4 * BASE, dv=5 * BASE, dg=6 * BASE,
              dbeta=7 * BASE, da_log=8 * BASE, ddt_bias=9 * BASE, d_initial_state=10 * BASE, workspace=16 * BASE,
              workspace_bytes=LARGE), **kw)
    b.fwd = _fwd(**(fwd or {}))
    return b


COMMON = [(dict(B=0), INVALID), (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(Hk=3), INVALID), (dict(Hk=-1), INVALID),
          (dict(qkv_dtype=2), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
          (dict(g=None), INVALID), (dict(beta=None), INVALID), (dict(a_log=None), INVALID),
          (dict(flags=kda.KDA_TEST_WAIT_TIMEOUT), INVALID), (dict(flags=1 << 20), INVALID),
          (dict(cu_seqlens=BASE, num_seqs=2), INVALID), (dict(cu_seqlens=BASE, B=1, num_seqs=0), INVALID),
          (dict(dk=96), UNSUPPORTED), (dict(dv=256), UNSUPPORTED), (dict(chunk=32), UNSUPPORTED),
          (dict(h_out=BASE), UNSUPPORTED), (dict(v_new_out=BASE), UNSUPPORTED), (dict(flags=kda.KDA_REUSE_PREP), UNSUPPORTED),
          (dict(flags=kda.KDA_SAFE_GATE), UNSUPPORTED), (dict(flags=kda.KDA_ALLOW_NEG_EIGVAL), UNSUPPORTED),
          (dict(T=1 << 30, H=128, Hk=1), UNSUPPORTED), (dict(T=(1 << 31) - 1), UNSUPPORTED),
          (dict(q=BASE + 2), ALIGNMENT), (dict(g=BASE + 4), ALIGNMENT), (dict(initial_state=BASE + 8), ALIGNMENT)]


@pytest.mark.parametrize("kw,want", COMMON + [
    (dict(out=None), INVALID), (dict(out=BASE + 4), ALIGNMENT), (dict(final_state=BASE + 4), ALIGNMENT),
    (dict(workspace=None), WORKSPACE), (dict(workspace=BASE + 16), ALIGNMENT)])
def test_fwd_refusals(lib, kw, want):
    assert lib.kda_gdn_chunk_fwd(ctypes.byref(_fwd(**kw)), None) == want
    assert lib.kda_gdn_chunk_fwd(None, None) == INVALID


@pytest.mark.parametrize("kw,want", COMMON)
def test_bwd_refuses_what_the_forward_does(lib, kw, want):
    assert lib.kda_gdn_chunk_bwd(ctypes.byref(_bwd(kw)), None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(dq=None), INVALID), (dict(dk=None), INVALID), (dict(dv=None), INVALID), (dict(dg=None), INVALID), (dict(dbeta=None), INVALID),
    (dict(d_out=3 * BASE), INVALID), (dict(d_out=4 * BASE), INVALID), (dict(d_out=5 * BASE), INVALID),
    (dict(d_out=BASE + 2), ALIGNMENT), (dict(d_initial_state=BASE + 4), ALIGNMENT), (dict(workspace=None), WORKSPACE),
    (dict(workspace=BASE + 128), ALIGNMENT)])
def test_bwd_refusals(lib, kw, want):
    assert lib.kda_gdn_chunk_bwd(ctypes.byref(_bwd(**kw)), None) == want
    assert lib.kda_gdn_chunk_bwd(None, None) == INVALID


def test_workspace_sizes(lib):
    for size, call, make in ((lib.kda_gdn_chunk_fwd_workspace_size, lib.kda_gdn_chunk_fwd, _fwd),
                             (lib.kda_gdn_chunk_bwd_workspace_size, lib.kda_gdn_chunk_bwd, _bwd)):
        need = size(ctypes.byref(make()))
        assert need > 0
        assert call(ctypes.byref(make(workspace_bytes=need - 1)), None) == WORKSPACE
    assert lib.kda_gdn_chunk_fwd_workspace_size(ctypes.byref(_fwd(dk=96))) == 0
    assert lib.kda_gdn_chunk_bwd_workspace_size(ctypes.byref(_bwd(dict(dk=96)))) == 0
    small, large = (lib.kda_gdn_chunk_fwd_workspace_size(ctypes.byref(_fwd(T=t))) for t in (100, 1000))
    assert small < large


def _step(**kw):
    return _fill(kda.kda_decode_args(), dict(N=3, T=1, H=4, dk=128, dv=128, qkv_dtype=kda.KDA_BF16, q=BASE, k=2 * BASE, v=3 * BASE,
                 g=4 * BASE, beta=5 * BASE, scale=0.1, eps=1e-6, out=6 * BASE, cache=7 * BASE, cache_dtype=kda.KDA_F32, num_rows=8,
                 row_stride_elems=4 * 128 * 128, idx=8 * BASE, idx_dtype=kda.KDA_I32, Hk=2), **kw)


@pytest.mark.parametrize("kw,want", [
    (dict(N=-1), INVALID), (dict(T=0), INVALID), (dict(H=0), INVALID), (dict(Hk=3), INVALID), (dict(qkv_dtype=9), INVALID),
    (dict(cache_dtype=9), INVALID), (dict(idx_dtype=2), INVALID), (dict(num_rows=0), INVALID),
    (dict(row_stride_elems=4 * 128 * 128 - 1), INVALID), (dict(flags=kda.KDA_GATE_IN_KERNEL), INVALID),
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(cache=None), INVALID), (dict(idx=None), INVALID),
    (dict(dk=32), UNSUPPORTED), (dict(dv=32), UNSUPPORTED), (dict(flags=kda.KDA_LAYOUT_HEAD_MAJOR), UNSUPPORTED),
    (dict(flags=kda.KDA_REUSE_PREP), UNSUPPORTED), (dict(N=1 << 30), UNSUPPORTED), (dict(N=0), 0)])
def test_step_refusals(lib, kw, want):
    assert lib.kda_gdn_recurrent_step(ctypes.byref(_step(**kw)), None) == want
    assert lib.kda_gdn_recurrent_step(None, None) == INVALID


LORA = dict(rows=10, n_in=64, n_out=32, rank=8, adapters=3, dtype=kda.KDA_BF16, x=BASE, a=2 * BASE, b=3 * BASE, idx=4 * BASE,
            idx_dtype=kda.KDA_I32, num_requests=5, scale=5 * BASE)


def _lora(**kw):
    return _fill(kda.kda_lora_args(), dict(LORA, y=6 * BASE, out=7 * BASE), **kw)


def _lora_bwd(**kw):
    return _fill(kda.kda_lora_bwd_args(), dict(LORA, d_out=6 * BASE, d_x_in=7 * BASE, d_x=8 * BASE, d_a=9 * BASE, d_b=10 * BASE,
                 workspace=16 * BASE, workspace_bytes=LARGE), **kw)


LORA_COMMON = [(dict(rows=-1), INVALID), (dict(n_in=0), INVALID), (dict(n_out=0), INVALID), (dict(rank=0), INVALID),
               (dict(adapters=0), INVALID), (dict(dtype=5), INVALID), (dict(idx_dtype=5), INVALID), (dict(num_requests=0), INVALID),
               (dict(num_requests=-1, rows=0), INVALID), (dict(num_requests=3), INVALID), (dict(x=None), INVALID),
               (dict(a=None), INVALID), (dict(b=None), INVALID), (dict(idx=None), INVALID), (dict(rank=129), UNSUPPORTED),
               (dict(adapters=65536), UNSUPPORTED), (dict(rows=1 << 31, num_requests=1), UNSUPPORTED),
               (dict(n_in=(1 << 31) - 1), UNSUPPORTED), (dict(n_out=(1 << 31) - 1), UNSUPPORTED), (dict(x=BASE + 2), ALIGNMENT),
               (dict(a=BASE + 8), ALIGNMENT), (dict(scale=BASE + 4), ALIGNMENT)]


@pytest.mark.parametrize("kw,want", LORA_COMMON + [
    (dict(y=None), INVALID), (dict(out=None), INVALID), (dict(out=BASE), INVALID), (dict(y=BASE + 2), ALIGNMENT), (dict(out=BASE + 2), ALIGNMENT),
    (dict(rows=0), 0), (dict(rows=0, num_requests=0), 0)])
def test_lora_refusals(lib, kw, want):
    assert lib.kda_lora(ctypes.byref(_lora(**kw)), None) == want
    assert lib.kda_lora(None, None) == INVALID


@pytest.mark.parametrize("kw,want", LORA_COMMON + [
    (dict(d_out=None), INVALID), (dict(d_x=BASE), INVALID), (dict(d_x=6 * BASE), INVALID), (dict(d_x=None, d_a=None, d_b=None), INVALID), (dict(d_out=BASE + 2), ALIGNMENT),
    (dict(d_x=BASE + 2), ALIGNMENT), (dict(d_a=BASE + 4), ALIGNMENT), (dict(workspace=None), WORKSPACE),
    (dict(workspace=BASE + 64), ALIGNMENT), (dict(adapters=65535, n_in=1 << 18, n_out=1 << 18), UNSUPPORTED)])
def test_lora_bwd_refusals(lib, kw, want):
    assert lib.kda_lora_bwd(ctypes.byref(_lora_bwd(**kw)), None) == want
    assert lib.kda_lora_bwd(None, None) == INVALID


def test_lora_workspace(lib):
    need = lib.kda_lora_bwd_workspace_size(ctypes.byref(_lora_bwd()))
    assert need > 0
    assert lib.kda_lora_bwd(ctypes.byref(_lora_bwd(workspace_bytes=need - 1)), None) == WORKSPACE
    assert lib.kda_lora_bwd_workspace_size(ctypes.byref(_lora_bwd(rank=129))) == 0


def _gdn(T=10, H=4, Hk=2, dk=128, dv=64, dtype=torch.bfloat16):
    return [torch.zeros(1, T, Hk, dk, dtype=dtype), torch.zeros(1, T, Hk, dk, dtype=dtype), torch.zeros(1, T, H, dv, dtype=dtype),
            torch.zeros(1, T, H), torch.zeros(1, T, H)]


def test_binding_chunk_refusals(lib):
    x = _gdn()
    for call in (kda.kda_gdn_chunk_fwd, lambda *a, **kw: kda.kda_gdn_chunk_bwd(*a, None, **kw)):
        with pytest.raises(ValueError, match="CUDA tensors"):
            call(*x)
        with pytest.raises(ValueError, match="without the channel axis"):
            call(*x[:3], torch.zeros(1, 10, 4, 128), x[4])
        with pytest.raises(ValueError, match="leading dims"):
            call(x[0][:, :9], *x[1:])
        with pytest.raises(ValueError, match="divide"):
            call(*_gdn(Hk=3))
        with pytest.raises(TypeError, match="one dtype"):
            call(x[0].float(), *x[1:])
        with pytest.raises(TypeError, match="fp32"):
            call(*x[:3], x[3].bfloat16(), x[4])
        with pytest.raises(ValueError, match="needs a_log"):
            call(*x, gate_in_kernel=True)
        with pytest.raises(ValueError, match="dt_bias"):
            call(*x, gate_in_kernel=True, a_log=torch.zeros(4), dt_bias=torch.zeros(4, 128))
        with pytest.raises(ValueError, match="initial_state"):
            call(*x, initial_state=torch.zeros(1, 4, 64, 128))
        with pytest.raises(ValueError, match="one token axis"):
            call(*x, cu_seqlens=torch.zeros(2, dtype=torch.int32))
        with pytest.raises(ValueError, match="cu_seqlens must"):
            call(*(t[0] for t in x), cu_seqlens=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="out must"):
        kda.kda_gdn_chunk_fwd(*x, out=torch.zeros(1, 10, 4, 64))
    with pytest.raises(ValueError, match="d_out must"):
        kda.kda_gdn_chunk_bwd(*x, torch.zeros(1, 10, 4, 64))


def test_binding_step_refusals(lib):
    x, cache, idx = _gdn(T=1), torch.zeros(3, 4, 128, 64), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensors"):
        kda.kda_gdn_recurrent_step(*x, cache, idx)
    with pytest.raises(ValueError, match="cache must"):
        kda.kda_gdn_recurrent_step(*x, cache.transpose(2, 3), idx)
    with pytest.raises(ValueError, match="dense"):
        kda.kda_gdn_recurrent_step(*x, torch.zeros(3, 4, 64, 128).transpose(2, 3), idx)
    with pytest.raises(ValueError, match="idx must"):
        kda.kda_gdn_recurrent_step(*x, cache, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(TypeError, match="int32 or int64"):
        kda.kda_gdn_recurrent_step(*x, cache, idx.short())
    with pytest.raises(TypeError, match="init_flags"):
        kda.kda_gdn_recurrent_step(*x, cache, idx, idx)
    with pytest.raises(ValueError, match="without the channel axis"):
        kda.kda_gdn_recurrent_step(*x[:3], torch.zeros(1, 1, 4, 128), x[4], cache, idx)


def test_binding_lora_refusals(lib):
    x, a, b, idx, y = (torch.zeros(6, 32), torch.zeros(3, 4, 32), torch.zeros(3, 16, 4), torch.zeros(2, dtype=torch.int32),
                       torch.zeros(6, 16))
    with pytest.raises(ValueError, match="CUDA tensors"):
        kda.kda_lora(x, a, b, idx, y)
    with pytest.raises(ValueError, match="CUDA tensors"):
        kda.kda_lora_bwd(y, x, a, b, idx)
    with pytest.raises(ValueError, match="do not go with"):
        kda.kda_lora(x, a, b[:, :, :3], idx, y)
    with pytest.raises(ValueError, match="y must"):
        kda.kda_lora(x, a, b, idx, y.bfloat16())
    with pytest.raises(TypeError, match="one dtype"):
        kda.kda_lora(x, a.bfloat16(), b, idx, y)
    with pytest.raises(ValueError, match="cannot be shared out"):
        kda.kda_lora(x, a, b, torch.zeros(4, dtype=torch.int32), y)
    with pytest.raises(ValueError, match="cu_seqlens must"):
        kda.kda_lora(x, a, b, idx, y, cu_seqlens=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="scale must"):
        kda.kda_lora(x, a, b, idx, y, scale=torch.zeros(2))
    with pytest.raises(TypeError, match="int32 or int64"):
        kda.kda_lora(x, a, b, idx.float(), y)
    with pytest.raises(TypeError, match="unsupported dtype"):
        kda.kda_lora(x.half(), a.half(), b.half(), idx, y.half())
    with pytest.raises(ValueError, match="no gradient"):
        kda.kda_lora_bwd(y, x, a, b, idx, want_dx=False, want_weights=False)
