"""The 8-bit layer's and the block norms' entry points reject bad arguments with
the documented status before touching a device; no call reaches a launch."""
import ctypes

import pytest
import torch

import activation_sparse_gemm_amd as lynx
from activation_sparse_gemm_amd import _abi

OK, NULL, SHAPE, ALIGN, WORKSPACE = range(5)
UNSUPPORTED = 6
A, B = 0x10000, 0x20000


@pytest.mark.parametrize("fn", ["lynx_quantize_fp8", "lynx_quantize_fp8_weight"])
@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), SHAPE), (dict(K=100), SHAPE), (dict(K=0), SHAPE), (dict(rows=1 << 25), SHAPE),
    (dict(rows=1 << 23, K=1 << 10), SHAPE), (dict(x=None), NULL), (dict(q=None), NULL),
    (dict(s=None), NULL), (dict(x=A + 2), ALIGN), (dict(q=A + 8), ALIGN), (dict(s=A + 4), ALIGN),
    (dict(rows=0), OK), (dict(rows=0, x=None), OK),
])
def test_quantize_validation(fn, kw, status):
    a = dict(x=A, rows=16, K=128, q=A, s=A) | kw
    assert getattr(_abi.lib(), fn)(a["x"], a["rows"], a["K"], a["q"], a["s"], None) == status


def test_workspace_bytes():
    ws = _abi.fp8_workspace_bytes
    # values and scale words (one per row and 512 channels), each rounded up to 256
    assert ws(4096, 12288, 3072) == 4096 * 3072 + 6 * 4096 * 4
    assert ws(333, 4096, 1472) == 490240 + 4096
    assert ws(9, 100, 4160) == 37632 + 512
    # few rows and few tiles are quantised inside the product
    assert ws(8, 100, 4096) == 0 and ws(1, 18432, 12288) == 0 and ws(16, 8191, 2048) == 0
    assert ws(300, 1024, 1024) == 0 and ws(4096, 64, 3072) == 0 and ws(17, 16, 64) == 0
    assert ws(8, 100, 4160) > 0 and ws(16, 8192, 2560) > 0 and ws(300, 1024, 2112) > 0
    assert ws(0, 16, 64) == 0 and ws(4, 16, 100) == 0 and ws(-1, 16, 64) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(K=96), SHAPE), (dict(M=-1), SHAPE), (dict(N=-1), SHAPE), (dict(M=1 << 20, N=1 << 12), SHAPE),
    (dict(x=None), NULL), (dict(wq=None), NULL), (dict(ws=None), NULL), (dict(y=None), NULL),
    (dict(x=A + 1), ALIGN), (dict(wq=A + 8), ALIGN), (dict(ws=A + 4), ALIGN), (dict(y=A + 2), ALIGN),
    (dict(M=17, K=4096, ws_=None), WORKSPACE), (dict(M=17, K=4096, n=17 * 4096 + 767), WORKSPACE),
    (dict(M=17, K=4096, ws_=B + 16), ALIGN),
    (dict(M=0), OK), (dict(N=0), OK),
])
def test_linear_validation(kw, status):
    a = dict(x=A, wq=A, ws=A, y=A, M=16, N=16, K=128, ws_=B, n=1 << 20) | kw
    f = _abi.lib().lynx_linear_fp8
    assert f(a["x"], a["wq"], a["ws"], a["y"], a["M"], a["N"], a["K"], a["ws_"], a["n"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(K=96), SHAPE), (dict(xq=None), NULL), (dict(xs=None), NULL), (dict(y=None), NULL),
    (dict(xq=A + 8), ALIGN), (dict(xs=A + 4), ALIGN), (dict(M=0), OK), (dict(N=0, y=None), OK),
])
def test_packed_validation(kw, status):
    a = dict(xq=A, xs=A, wq=A, ws=A, y=A, M=16, N=16, K=128) | kw
    f = _abi.lib().lynx_linear_fp8_packed
    assert f(a["xq"], a["xs"], a["wq"], a["ws"], a["y"], a["M"], a["N"], a["K"], None) == status


def norm(**kw):
    d = dict(x=A, h=A, M=16, C=64, samples=1, residual_scale=1.0, eps=1e-6, norm=1) | kw
    return _abi.lib().lynx_block_norm(ctypes.byref(_abi.Norm(**d)), None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), SHAPE), (dict(M=(1 << 23) + 1), SHAPE), (dict(C=0), SHAPE), (dict(C=12), SHAPE),
    (dict(C=16392), SHAPE), (dict(samples=0), SHAPE), (dict(samples=3), SHAPE),
    (dict(gate_stride=4), SHAPE), (dict(shift_stride=-8), SHAPE), (dict(norm=3), SHAPE),
    (dict(post_norm=-1), SHAPE), (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE),
    (dict(C=72, h=None, q=A, q_scale=A), SHAPE),
    (dict(x=None), NULL), (dict(h=None), NULL), (dict(q=A, q_scale=A), NULL),
    (dict(h=None, q=A), NULL), (dict(q_scale=A), NULL), (dict(y=A), NULL), (dict(x_out=A), NULL),
    (dict(gate=A), NULL), (dict(post_norm=1), NULL), (dict(y=A, x_out=A, post_weight=A), NULL),
    (dict(norm=0, h=None), NULL), (dict(norm=0, y=A, x_out=A), NULL),
    (dict(norm=0, h=None, y=A, x_out=A, scale=A), NULL),
    (dict(x=A + 8), ALIGN), (dict(h=A + 2), ALIGN), (dict(scale=A + 2), ALIGN),
    (dict(y=A, x_out=A + 4), ALIGN), (dict(M=0, x=None, h=None), OK),
])
def test_norm_validation(kw, status):
    assert norm(**kw) == status


def test_norm_null_descriptor():
    assert _abi.lib().lynx_block_norm(None, None) == NULL


@pytest.mark.skipif(torch.cuda.is_available(), reason="valid fake pointers must not reach a launch")
def test_valid_arguments_reach_the_device_check():
    L = _abi.lib()
    assert L.lynx_quantize_fp8(A, 16, 64, A, A, None) == UNSUPPORTED
    assert L.lynx_linear_fp8_packed(A, A, A, A, A, 1, 1, 64, None) == UNSUPPORTED
    assert norm() == UNSUPPORTED
    assert norm(norm=0, h=None, y=A, x_out=A, gate=A) == UNSUPPORTED
    assert norm(y=A, x_out=A, h=None, q=A, q_scale=A, post_norm=2, C=16384) == UNSUPPORTED


def test_python_refusals():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    for call in (lambda: lynx.quantize_fp8(x), lambda: lynx.quantize_fp8_weight(x),
                 lambda: lynx.norm_modulate(x), lambda: lynx.residual_norm(x, x),
                 lambda: lynx.linear_fp8(x, x, x), lambda: lynx.linear_fp8_packed(x, x, x, x)):
        with pytest.raises(ValueError, match="device tensor"):
            call()
    with pytest.raises(ValueError, match="needs a norm"):
        lynx.norm_modulate(x, norm=None)
    with pytest.raises(ValueError, match="needs y"):
        lynx.residual_norm(x, None)
    with pytest.raises(ValueError, match="matrix"):
        lynx.quantize_fp8(x[0])
