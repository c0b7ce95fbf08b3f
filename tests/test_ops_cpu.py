"""Refusals of the operators around the linears that need no GPU, and the tests' own e4m3 rounding."""
import ctypes
import math

import numpy as np
import pytest
import torch

import ops_ref as R

P = ctypes.c_void_p
d, odd4, odd2 = P(1 << 20), P((1 << 20) + 4), P((1 << 20) + 2)


@pytest.fixture(scope="module")
def lib():
    from w4a8_block_quantized_gb300 import binding, build
    build.build()
    return binding.load()


def b():
    from w4a8_block_quantized_gb300 import binding
    return binding


def test_e4m3_rounding_agrees_with_every_code():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy().astype(np.float64)
    codes = codes[np.isfinite(codes)]
    assert np.array_equal(R.e4m3(codes), codes)
    v = np.random.default_rng(0).standard_normal(20000).astype(np.float32) * np.float32(30)
    v = np.concatenate([v, v * np.float32(1e-4)])
    assert np.array_equal(R.e4m3(v), torch.from_numpy(v).to(torch.float8_e4m3fn).double().numpy())


def norm(lib, x=d, res=d, g=d, eps=1e-6, dt=1, out=d, q=d, s=d, rs=d, M=4, K=128):
    return lib.w4a8_rmsnorm_quant(x, res, g, eps, dt, out, q, s, rs, M, K, None)


def norm8(lib, x=d, res=d, g=d, eps=1e-6, dt=1, out=d, q=d, s=d, M=4, K=128):
    return lib.w4a8_rmsnorm_quant_fp8(x, res, g, eps, dt, out, q, s, M, K, None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), -1), (dict(g=None), -1), (dict(q=None), -1), (dict(s=None), -1), (dict(M=-1), -1), (dict(dt=2), -1),
    (dict(dt=-1), -1), (dict(eps=0.0), -1), (dict(eps=-1.0), -1), (dict(eps=math.inf), -1), (dict(eps=math.nan), -1),
    (dict(res=None), -1), (dict(K=0), -3), (dict(K=100), -3), (dict(K=-64), -3), (dict(M=1 << 31), -3), (dict(x=odd4), -2),
    (dict(res=odd4), -2), (dict(out=odd4), -2), (dict(g=odd4), -2), (dict(q=odd4), -2), (dict(s=odd2), -2)])
def test_norm_refusals(lib, kw, want):
    assert norm(lib, **kw) == want
    assert norm8(lib, **kw) == want


def test_norm_refusals_of_one_form(lib):
    assert norm(lib, rs=None) == b().W4A8_ERR_ARG
    assert norm(lib, rs=odd2) == b().W4A8_ERR_ALIGN
    assert norm(lib, K=96) == b().W4A8_ERR_SHAPE      # whole 64-blocks
    assert norm8(lib, K=40) == b().W4A8_ERR_SHAPE     # whole 16-byte rows
    need = lib.w4a8_prepared_activations_bytes(4, 128)
    call = lambda act, n: lib.w4a8_rmsnorm_prepare(d, d, d, 1e-6, 1, d, act, n, 4, 128, None)  # noqa: E731
    assert call(None, need) == b().W4A8_ERR_ARG
    assert call(odd4, need) == b().W4A8_ERR_ALIGN
    assert call(d, need - 1) == b().W4A8_ERR_WORKSPACE
    # an empty problem reads no pointer
    assert norm(lib, M=0, x=None, q=None) == b().W4A8_OK and norm8(lib, M=0, x=None) == b().W4A8_OK


@pytest.mark.parametrize("kw,want", [
    (dict(g=None), -1), (dict(u=None), -1), (dict(q=None), -1), (dict(s=None), -1), (dict(M=-1), -1), (dict(dt=7), -1),
    (dict(ld=64), -3), (dict(ld=1 << 31), -3), (dict(K=0), -3), (dict(K=130), -3), (dict(g=odd4), -2), (dict(u=odd4), -2),
    (dict(ld=260), -2), (dict(ld=258, dt=0), -2), (dict(q=odd4), -2), (dict(s=odd2), -2)])
def test_swiglu_refusals(lib, kw, want):
    a = dict(g=d, u=d, ld=256, dt=1, q=d, s=d, M=4, K=128)
    a.update(kw)
    assert lib.w4a8_swiglu_quant(a["g"], a["u"], a["ld"], a["dt"], a["q"], a["s"], d, a["M"], a["K"], None) == want
    assert lib.w4a8_swiglu_quant_fp8(a["g"], a["u"], a["ld"], a["dt"], a["q"], a["s"], a["M"], a["K"], None) == want


def test_swiglu_prepare_and_quant_refusals(lib):
    need = lib.w4a8_prepared_activations_bytes(4, 128)
    assert lib.w4a8_swiglu_prepare(d, d, 128, 1, d, need - 1, 4, 128, None) == b().W4A8_ERR_WORKSPACE
    assert lib.w4a8_swiglu_prepare(d, d, 128, 1, None, need, 4, 128, None) == b().W4A8_ERR_ARG
    assert lib.w4a8_quant_fp8(None, 0, d, d, 4, 128, None) == b().W4A8_ERR_ARG
    assert lib.w4a8_quant_fp8(odd4, 0, d, d, 4, 128, None) == b().W4A8_ERR_ALIGN
    assert lib.w4a8_quant_fp8(d, 0, d, d, 4, 120, None) == b().W4A8_ERR_SHAPE
    assert lib.w4a8_quant_fp8(d, 3, d, d, 4, 128, None) == b().W4A8_ERR_ARG


@pytest.mark.parametrize("kw,want", [
    (dict(a=None), -1), (dict(sa=None), -1), (dict(w=None), -1), (dict(sw=None), -1), (dict(y=None), -1), (dict(dt=2), -1),
    (dict(M=-1), -1), (dict(N=-1), -1), (dict(K=0), -3), (dict(K=24), -3), (dict(M=1 << 31), -3), (dict(N=1 << 31), -3),
    (dict(M=1 << 30, N=1 << 30), -3), (dict(a=odd4), -2), (dict(w=odd4), -2), (dict(y=odd4), -2), (dict(sa=odd2), -2),
    (dict(sw=odd2), -2), (dict(bias=odd2), -2)])
def test_fp8_linear_refusals(lib, kw, want):
    a = dict(a=d, sa=d, w=d, sw=d, bias=None, y=d, dt=0, M=4, N=8, K=128)
    a.update(kw)
    assert lib.w4a8_fp8_linear(*(a[k] for k in ("a", "sa", "w", "sw", "bias", "y", "dt", "M", "N", "K")), None) == want


def test_fp8_linear_empty(lib):
    assert lib.w4a8_fp8_linear(None, None, None, None, None, None, 0, 0, 8, 128, None) == b().W4A8_OK
    assert lib.w4a8_fp8_linear(None, None, None, None, None, None, 1, 8, 0, 128, None) == b().W4A8_OK


def test_binding_rejects_host_tensors():
    x, w = torch.zeros((4, 128)), torch.zeros(128)
    q8 = torch.zeros((4, 128)).to(torch.float8_e4m3fn)
    s = torch.zeros((1, 4))
    for call in (lambda: b().rmsnorm_quant(x, w, 1e-6), lambda: b().rmsnorm_prepare(x, w, 1e-6),
                 lambda: b().rmsnorm_quant_fp8(x, w, 1e-6), lambda: b().swiglu_quant(x, x),
                 lambda: b().swiglu_prepare(x, x), lambda: b().swiglu_quant_fp8(x, x), lambda: b().quant_fp8(x),
                 lambda: b().fp8_linear(q8, s, q8, s)):
        with pytest.raises(TypeError, match="CUDA tensor"):
            call()
