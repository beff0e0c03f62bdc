"""The entry points of rotary positions and attention reject bad arguments with the documented
status before touching a device; no call reaches a launch."""
import ctypes

import pytest
import torch

import activation_sparse_gemm_amd as lynx
from activation_sparse_gemm_amd import _abi

OK, NULL, SHAPE, ALIGN, WORKSPACE = range(5)
UNSUPPORTED = 6
A, B = 0x10000, 0x20000
NAN, INF = float("nan"), float("inf")


def rotary(axis_dims=(16, 24, 24), **kw):
    d = dict(q=A, k=A, q_weight=A, k_weight=A, positions=A, q_out=B, k_out=B, tokens=5, q_heads=4, k_heads=2,
             head_dim=64, q_stride=512, q_head_stride=64, k_stride=512, k_head_stride=64, q_out_stride=256,
             q_out_head_stride=64, k_out_stride=128, k_out_head_stride=64, theta=1e4, axes=len(axis_dims), norm=1,
             eps=1e-6) | kw
    s = _abi.Rotary(**d)
    for i, n in enumerate(axis_dims):
        s.axis_dims[i] = n
    return _abi.lib().lynx_qk_rotary(ctypes.byref(s), None)


@pytest.mark.parametrize("kw,status", [
    (dict(head_dim=0), SHAPE), (dict(head_dim=60), SHAPE), (dict(head_dim=264), SHAPE), (dict(head_dim=56), SHAPE),
    (dict(axis_dims=()), SHAPE), (dict(axes=5), SHAPE), (dict(axis_dims=(16, 23, 24)), SHAPE),
    (dict(axis_dims=(16, 0, 24)), SHAPE), (dict(axis_dims=(-2, 4)), SHAPE), (dict(axis_dims=(40, 26)), SHAPE),
    (dict(axis_dims=(2 ** 30, 2 ** 30, 2 ** 30, 2 ** 30)), SHAPE),
    (dict(tokens=-1), SHAPE), (dict(tokens=(1 << 24) + 1), SHAPE), (dict(tokens=1 << 24, q_heads=200), SHAPE),
    (dict(q_heads=0), SHAPE), (dict(q_heads=1025), SHAPE), (dict(k_heads=-1), SHAPE), (dict(k_heads=1025), SHAPE),
    (dict(theta=0.0), SHAPE), (dict(theta=-2.0), SHAPE), (dict(theta=NAN), SHAPE), (dict(theta=INF), SHAPE),
    (dict(pairs=2), SHAPE), (dict(ladder=-1), SHAPE), (dict(norm=2), SHAPE), (dict(norm=-1), SHAPE),
    (dict(eps=-1.0), SHAPE), (dict(eps=NAN), SHAPE), (dict(q_stride=4), SHAPE), (dict(k_stride=-8), SHAPE),
    (dict(q_head_stride=1), SHAPE), (dict(k_out_head_stride=-64), SHAPE),
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(positions=None), NULL), (dict(q_out=None), NULL),
    (dict(k_out=None), NULL), (dict(k_heads=0), NULL), (dict(norm=0), NULL),
    (dict(norm=0, q_weight=None), NULL),
    (dict(q=A + 8), ALIGN), (dict(k=A + 2), ALIGN), (dict(q_weight=A + 8), ALIGN), (dict(positions=A + 4), ALIGN),
    (dict(k_out=B + 8), ALIGN),
    (dict(tokens=0), OK), (dict(tokens=0, q=None, k=None), OK),
])
def test_rotary_validation(kw, status):
    assert rotary(**kw) == status


ATTN = dict(q=A, k=A, v=A, out=B, batch=2, tokens_q=64, tokens_k=64, heads=4, kv_heads=2, head_dim=64,
            q_batch_stride=8192, q_stride=256, q_head_stride=64, k_batch_stride=4096, k_stride=128, k_head_stride=64,
            v_batch_stride=4096, v_stride=128, v_head_stride=64, out_batch_stride=8192, out_stride=256,
            out_head_stride=64, scale=0.125)
PREFIX = dict(prefix_tokens=300, prefix_k=A, prefix_v=A, prefix_k_stride=128, prefix_k_head_stride=64,
              prefix_v_stride=128, prefix_v_head_stride=64)
CUT = dict(batch=1, tokens_q=1, tokens_k=9000, heads=1, kv_heads=1)


def attn(ws=None, n=0, **kw):
    return _abi.lib().lynx_attention(ctypes.byref(_abi.Attn(**(ATTN | kw))), ws, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(head_dim=0), SHAPE), (dict(head_dim=60), SHAPE), (dict(head_dim=136), SHAPE),
    (dict(heads=0), SHAPE), (dict(heads=5), SHAPE), (dict(heads=1026), SHAPE), (dict(kv_heads=0), SHAPE),
    (dict(kv_heads=8), SHAPE), (dict(batch=0), SHAPE), (dict(batch=(1 << 16) + 1), SHAPE),
    (dict(tokens_q=-2), SHAPE), (dict(tokens_k=(1 << 26) + 2), SHAPE), (dict(prefix_tokens=-1), SHAPE),
    (dict(tokens_q=1 << 26, heads=16), SHAPE), (dict(tokens_q=65), SHAPE), (dict(tokens_k=63), SHAPE),
    (dict(scale=0.0), SHAPE), (dict(scale=-1.0), SHAPE), (dict(scale=NAN), SHAPE), (dict(scale=INF), SHAPE),
    (dict(q_stride=4), SHAPE), (dict(k_stride=-8), SHAPE), (dict(out_head_stride=1), SHAPE),
    (dict(q_batch_stride=7), SHAPE), (dict(k_stride=56), SHAPE), (dict(v_stride=0), SHAPE),
    (dict(k_stride=1 << 24), SHAPE), (dict(v_stride=1 << 23), SHAPE),
    (dict(batch=1 << 16, tokens_q=1 << 16, heads=64, kv_heads=64), SHAPE), (PREFIX | dict(prefix_v_stride=0), SHAPE),
    (PREFIX | dict(prefix_k_head_stride=4), SHAPE),
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(out=None), NULL),
    (dict(cu_q=A), NULL), (dict(cu_k=A), NULL), (dict(prefix_k=A), NULL), (PREFIX | dict(prefix_v=None), NULL),
    (dict(q=A + 8), ALIGN), (dict(v=A + 2), ALIGN), (dict(out=B + 8), ALIGN), (dict(cu_q=A + 2, cu_k=A), ALIGN),
    (dict(lse=B + 1), ALIGN), (PREFIX | dict(prefix_k=A + 8), ALIGN),
    (CUT, WORKSPACE), (CUT | dict(ws=B, n=16), WORKSPACE), (CUT | dict(ws=B + 16, n=1 << 30), ALIGN),
    (dict(tokens_q=0), OK), (dict(tokens_q=0, q=None, out=None), OK),
])
def test_attention_validation(kw, status):
    assert attn(**kw) == status


def test_bases_whose_frequencies_pass_64_bits():
    # theta^(-2 j / n) reaches 1 / theta nearly; infinite ones made NaN of position 0
    assert rotary(theta=5e-324) == SHAPE and rotary(theta=5e-324, tokens=0) == SHAPE
    assert rotary(theta=2.0 ** -1022, tokens=0) == OK and rotary(theta=1e308, tokens=0) == OK


def test_scales_that_pass_fp32_with_log2_e():
    # above 2^128 / log2(e) = 2^127.47 every score that is 0 would become NaN
    for scale in (2.0 ** 127, 3.4e38):
        assert attn(scale=scale) == SHAPE
    assert attn(scale=2.0 ** 127, tokens_q=0) == SHAPE
    assert attn(scale=2.0 ** 127 * (1 - 2.0 ** -24), tokens_q=0) == OK and attn(scale=2.0 ** -149, tokens_q=0) == OK


def test_null_descriptors():
    L = _abi.lib()
    assert L.lynx_qk_rotary(None, None) == NULL
    assert L.lynx_attention(None, None, 0, None) == NULL
    assert L.lynx_attention_workspace_bytes(None) == 0


def test_attention_workspace():
    f = lynx.attention_workspace_bytes
    assert f(1, 4608, 4608, 24, 24, 128) == 0          # tiles enough: nothing is cut
    assert f(1, 1, 9000, 1, 1, 64) > 0
    assert f(4, 4, 4, 1, 1, 64, prefix_tokens=1) > 0   # a prefix of its own is joined
    assert f(0, 4, 4, 1, 1, 64) == 0 and f(1, 4, 4, 3, 2, 64) == 0 and f(1, 4, 4, 1, 1, 60) == 0
    sizes = (1, 64, 1 << 17, 8, 8, 128)                # as the call is: causal ones are cut otherwise
    assert all(f(*sizes, causal=c) > 0 for c in (False, True))
    for packed in (False, True):                       # never past a GiB for the sake of uneven lengths
        for tq, tk in ((1, 1 << 26), (64, 1 << 20), (4096, 1 << 20), (1 << 16, 1 << 20)):
            assert f(1, tq, tk, 32, 8, 128, packed=packed) <= 1 << 30


def test_a_row_has_as_many_partial_results_as_pieces_of_the_prefix():
    # 70000 keys are 547 tiles of 128; at most 128 pieces of whole tiles are 110 of 5, and the
    # tokens' own keys are one more.  What is not written must not be there to be joined.
    rows, slots, D = 2 * 8, 110 + 1, 128
    up = lambda n: (n + 255) // 256 * 256
    want = up(rows * slots * D * 4) + up(rows * slots * 16) + up(rows * 4)
    for packed in (False, True):
        assert lynx.attention_workspace_bytes(2, 2, 20, 8, 1, D, 70000, packed, True) == want


@pytest.mark.skipif(torch.cuda.is_available(), reason="valid fake pointers must not reach a launch")
def test_valid_arguments_reach_the_device_check():
    assert rotary() == UNSUPPORTED
    assert rotary(k=None, k_out=None, k_weight=None, k_heads=0) == UNSUPPORTED
    assert rotary(norm=0, q_weight=None, k_weight=None, axis_dims=(2,)) == UNSUPPORTED
    assert attn() == UNSUPPORTED
    assert attn(tokens_k=0, k=None, v=None) == UNSUPPORTED
    assert attn(cu_q=A, cu_k=A + 4, tokens_q=63, lse=B + 4) == UNSUPPORTED
    assert attn(ws=B, n=1 << 30, **PREFIX) == UNSUPPORTED


def test_python_refusals():
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    pos = torch.zeros((4, 1), dtype=torch.int32)
    for call in (lambda: lynx.qk_rotary(x, x, pos, (64,)), lambda: lynx.attention(x, x, x)):
        with pytest.raises(ValueError, match="device tensor"):
            call()
    with pytest.raises(ValueError, match="3 dimensions"):
        lynx.qk_rotary(x[0], x, pos, (64,))
    with pytest.raises(ValueError, match="3 or 4 dimensions"):
        lynx.attention(x[0], x, x)
