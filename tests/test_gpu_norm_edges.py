"""The block norms where single values decide: parameters and rows that are not
finite, rows whose squares overflow, and outputs at the low end of the 8-bit scales.
"""
import numpy as np
import pytest
import torch

import activation_sparse_gemm_amd as lynx
from oracle import block_oracle as bo
from tests.gpu_util import host_f64, say
from tests.test_gpu_norm import bf

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def ordinary(M, C, seed, f32=False):
    """Values between 1/4 and 4 of either sign: no zeros, no large spread."""
    rng = np.random.default_rng(seed)
    v = rng.choice([-1.0, 1.0], (M, C)) * np.exp2(rng.uniform(-2, 2, (M, C)))
    if f32:
        return torch.from_numpy(v.astype(np.float32)).cuda()
    return bf(v)[0]


def parameter(rows, C, seed):
    return ordinary(rows, C, seed)


def u8(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


# ---- parameters that are infinite --------------------------------------------------

@pytest.mark.parametrize("post", [None, "rms", "layer"])
@pytest.mark.parametrize("f32", [False, True])
def test_infinite_gate_without_a_bias(post, f32):
    """gate z is infinite where the gate is, with z's sign: an absent bias is no term."""
    M, C = 12, 640
    x, y, gate = ordinary(M, C, 1, f32), ordinary(M, C, 2), parameter(2, C, 3)
    ref, _ = lynx.residual_norm(x, y, gate=gate, post_norm=post)
    gate[0, 7], gate[1, 600] = INF, -INF
    say(f"infinite gate post={post} f32={f32}")
    got, _ = lynx.residual_norm(x, y, gate=gate, post_norm=post)
    z = host_f64(y)
    if post == "layer":
        z = z - z.mean(1, keepdims=True)
    got, want = host_f64(got), host_f64(ref)
    want[:6, 7] = INF * z[:6, 7]
    want[6:, 600] = -INF * z[6:, 600]
    assert np.array_equal(got, want)


@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("shift", [False, True])
def test_infinite_scale_without_a_bias(norm, shift):
    M, C = 12, 640
    x, scale = ordinary(M, C, 4), parameter(2, C, 5)
    kw = dict(norm=norm, shift=parameter(2, C, 6) if shift else None)
    ref = host_f64(lynx.norm_modulate(x, scale=scale, **kw))
    refq, refs = (u8(t) for t in lynx.norm_modulate(x, scale=scale, fp8=True, **kw))
    scale[0, 7], scale[1, 600] = INF, -INF
    say(f"infinite scale {norm} shift={shift}")
    t = host_f64(x)
    if norm == "layer":
        t = t - t.mean(1, keepdims=True)
    ref[:6, 7] = INF * t[:6, 7]
    ref[6:, 600] = -INF * t[6:, 600]
    assert np.array_equal(host_f64(lynx.norm_modulate(x, scale=scale, **kw)), ref)
    # in 8 bits the blocks that hold an infinity, and no others
    q, s = (u8(t) for t in lynx.norm_modulate(x, scale=scale, fp8=True, **kw))
    bad = np.zeros((M, 5), dtype=bool)
    bad[:6, 0] = bad[6:, 4] = True
    byte, refb = (v.transpose(1, 0, 2).reshape(M, -1)[:, :5] for v in (s, refs))
    assert np.array_equal(byte, np.where(bad, 255, refb))
    same = ~bad.repeat(128, 1)
    assert np.array_equal(q[same], refq[same])


# ---- rows that are not finite ------------------------------------------------------

SIZES = [64, 640, 2048, 4096, 8200]   # 1, 2, 4 and 8 waves a row, and 3 vectors a lane
BAD = [1, 2, 3, 5, 6]                 # rows of spoil() that a norm makes NaN


def spoil(t):
    """Rows with an infinity, a NaN, one value and many values whose squares pass fp32's range;
    row 7 is large and in range."""
    C = t.shape[1]
    t[1, C // 3], t[2, C - 1], t[3, 5] = INF, -INF, NAN
    t[5, C // 2] = 3e19
    t[6] *= 2.0 ** 64
    t[7, 9] = 2.0 ** 60
    return t


def whole_row(t, rows):
    """The rows of t that are NaN throughout are these, and the others are finite."""
    want = torch.zeros(t.shape, dtype=torch.bool, device="cuda")
    want[rows] = True
    return bool(torch.equal(torch.isnan(t), want)) and bool(torch.isfinite(t[~want]).all())


@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("C", SIZES)
def test_a_row_that_is_not_finite_becomes_nan(C, f32, norm):
    x = ordinary(9, C, 1, f32)
    ref = lynx.norm_modulate(x, norm)
    x = spoil(x)
    say(f"non-finite rows {norm} C={C} f32={f32}")
    h = lynx.norm_modulate(x, norm)
    assert whole_row(h, BAD)
    same = [0, 4, 8]
    assert torch.equal(h[same].view(torch.int16), ref[same].view(torch.int16))
    if C % 64 == 0:
        s = u8(lynx.norm_modulate(x, norm, fp8=True)[1])
        kb = -(-C // 128)
        byte = s.transpose(1, 0, 2).reshape(9, -1)[:, :kb]
        assert (byte[BAD] == 255).all() and not (np.delete(byte, BAD, 0) == 255).any()


@pytest.mark.parametrize("post", [None, "rms", "layer"])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("C", SIZES)
def test_a_branch_that_is_not_finite(C, f32, post):
    """A post norm makes all of x' NaN; without one x' holds the branch's value in its channel."""
    x, y = ordinary(9, C, 1, f32), spoil(ordinary(9, C, 2))
    say(f"non-finite branch {post} C={C} f32={f32}")
    for norm in (None, "rms", "layer"):
        xo, h = lynx.residual_norm(x, y, post_norm=post, norm=norm)
        if post:
            assert whole_row(xo, BAD)
        else:
            assert torch.equal(torch.isfinite(xo), torch.isfinite(y))
            assert torch.equal(torch.isnan(xo), torch.isnan(y))
        if norm:
            assert whole_row(h, BAD)
