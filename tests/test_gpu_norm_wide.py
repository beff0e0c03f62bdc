"""The block norms on rows of more than 8192 channels, where a lane holds three or four
vectors of eight, against the fp64 oracle.

Tolerances as in test_gpu_norm.py: a lane adds up to 32 values, the tree over 512 lanes
takes 9 steps, products, the mean and the root a few roundings more, fewer than 64 in
all; 2^-17 of the terms' magnitudes is 128 of 2^-24.  The oracle is evaluated on a
sample of the rows (a row's result depends on no other row) and every row is checked
for values that were not written.
"""
import numpy as np
import pytest
import torch

import activation_sparse_gemm_amd as lynx
import tests.gpu_util as gu
from oracle import block_oracle as bo
from tests.gpu_util import host_f64, say
from tests.test_gpu_norm import E8M0, FP8, check_fp8, close

pytestmark = pytest.mark.gpu


def randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def heavy(g, M, C):
    """A normal value times a log-normal factor of its channel, a few channels far above."""
    c = randn(g, C).exp() * torch.where(torch.rand((C,), generator=g, device="cuda") < 0.01, 20.0, 1.0)
    return randn(g, M, C) * c


def sample(M, B):
    """First and last rows, those on both sides of a sample's border, and some between."""
    rows = {0, 1, 2, M - 2, M - 1} | set(np.random.default_rng(M).integers(0, M, 12).tolist())
    for b in range(1, B):
        rows |= {b * (M // B) - 2, b * (M // B) - 1, b * (M // B), b * (M // B) + 1}
    return np.array(sorted(r for r in rows if 0 <= r < M))


def case(M, C, B, f32, branch, post, norm, affine, seed):
    """(x, arguments on the device)"""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    bf16 = torch.bfloat16
    x = heavy(g, M, C) if f32 else heavy(g, M, C).to(bf16)
    kw = {}
    # shift, scale and gate of a sample side by side, as a modulation projection writes them
    mod = (0.3 * randn(g, B, 3, C)).to(bf16)
    if branch:
        kw.update(y=heavy(g, M, C).to(bf16), gate=mod[:, 2], post_norm=post, post_eps=1e-5,
                  residual_scale=0.5 if f32 else 1.0)
        if post and affine:
            kw.update(post_weight=(1 + 0.2 * randn(g, C)).to(bf16), post_bias=(0.2 * randn(g, C)).to(bf16))
    kw["norm"] = norm
    if norm:
        kw.update(shift=mod[:, 0], scale=mod[:, 1], eps=1e-6)
        if affine:
            kw.update(weight=(1 + 0.2 * randn(g, C)).to(bf16), bias=(0.2 * randn(g, C)).to(bf16))
    return x, kw


def reference(x, kw, rows, B):
    """x', its magnitudes, h and its magnitudes of the sampled rows."""
    at = torch.from_numpy(rows).cuda()
    per = at // (x.shape[0] // B)
    f = {k: v for k, v in kw.items() if not torch.is_tensor(v)}
    for k, v in kw.items():
        if torch.is_tensor(v):
            pick = v[at] if k == "y" else v[per] if v.dim() == 2 else v
            f[k] = host_f64(pick)
    return bo.block_norm(host_f64(x[at]), **f)


WIDE = [  # C: the first of three vectors a lane, a ragged one, three full, the first of four, four full
    (1030, 8200, 2, False), (1030, 9216, 2, True), (6, 12288, 3, True), (1030, 12288, 2, False),
    (1030, 12296, 2, True), (1030, 16384, 2, False), (5, 16376, 1, True), (2050, 16384, 2, True)]


def check(M, C, B, f32, branch, post, norm, affine, fp8, label):
    x, kw = case(M, C, B, f32, branch, post, norm, affine, M + C)
    say(label)
    out = None
    if norm:
        out = gu.nan_bf16((M, C)) if not fp8 else (
            torch.full((M, C), 0xFF, dtype=torch.uint8, device="cuda").view(FP8),
            torch.full(((C + 511) // 512, M, 4), 0xAA, dtype=torch.uint8, device="cuda").view(E8M0))
    x_out = torch.full_like(x, float("nan"))
    if branch:
        _, h = lynx.residual_norm(x, fp8=fp8, x_out=x_out, out=out, **kw)
    else:
        h = lynx.norm_modulate(x, fp8=fp8, out=out, **kw)
    torch.cuda.synchronize()
    rows = sample(M, B)
    at = torch.from_numpy(rows).cuda()
    u, umag, hr, hmag = reference(x, kw, rows, B)
    if branch:
        assert bool(torch.isfinite(x_out).all()), label
        # without a post-norm there is no sum in x'
        close(host_f64(x_out[at]), u, umag, 2.0 ** -24 if f32 else 2.0 ** -8, label + " x'",
              2.0 ** -17 if post else 2.0 ** -22)
    if norm and fp8:
        q, s = h[0].view(torch.uint8), h[1].view(torch.uint8)
        assert not bool((q & 0x7F == 0x7F).any()) and not bool((s >= 0xAA).any()), label
        check_fp8((q[at], s[:, at].contiguous()), hr, hmag, label)
    elif norm:
        assert bool(torch.isfinite(h).all()), label
        close(host_f64(h[at]), hr, hmag, 2.0 ** -8, label + " h")


@pytest.mark.parametrize("post,norm", [(None, "rms"), ("rms", "layer"), ("layer", None), ("layer", "rms")])
@pytest.mark.parametrize("M,C,B,f32", WIDE)
def test_wide_residual_norm(M, C, B, f32, post, norm):
    check(M, C, B, f32, True, post, norm, post != norm, False,
          f"wide residual_norm {post} {norm} {M}x{C} B={B} f32={f32}")


@pytest.mark.parametrize("M,C,B,f32", [w for w in WIDE if w[1] % 64 == 0])
def test_wide_residual_norm_to_8_bits(M, C, B, f32):
    check(M, C, B, f32, True, "rms", "layer", f32, True, f"wide residual_norm fp8 {M}x{C} B={B} f32={f32}")


@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("M,C,B,f32", [(1030, 8200, 2, False), (1030, 12288, 2, True), (7, 12296, 1, False),
                                       (2050, 16384, 2, False)])
def test_wide_norm_modulate(M, C, B, f32, norm):
    check(M, C, B, f32, False, None, norm, True, C % 64 == 0 and norm == "rms",
          f"wide norm_modulate {norm} {M}x{C} B={B} f32={f32}")


@pytest.mark.parametrize("C,f32", [(8200, True), (16384, False), (16384, True)])
def test_wide_in_place_and_two_streams(C, f32):
    """x_out may be x; calls on two streams at once and graph replays give the same bytes."""
    M = 1030
    x, kw = case(M, C, 2, f32, True, "rms", "layer", True, 3)
    say(f"wide in place C={C} f32={f32}")
    ref_x, ref_h = lynx.residual_norm(x, **kw)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for st in streams:
        with torch.cuda.stream(st):
            outs += [lynx.residual_norm(x, **kw) for _ in range(2)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, ref_x) and torch.equal(b, ref_h) for a, b in outs)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gx, gh = lynx.residual_norm(x, **kw)
    for i in range(3):
        gx.fill_(0)
        gh.fill_(0)
        lynx.residual_norm(x, **kw)
        torch.cuda.synchronize()
        say(f"wide graph replay {i}")
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(gx, ref_x) and torch.equal(gh, ref_h)
    xi, hi = lynx.residual_norm(x, x_out=x, **kw)
    assert xi is x and torch.equal(xi, ref_x) and torch.equal(hi, ref_h)
