"""The 8-bit product and the norms' 8-bit output at both ends of the block scales.

The product of two scales is taken in the result's fp32 sums: with ones in both
operands every sum is a power of two times K, so the results below are exact.
"""
import numpy as np
import pytest
import torch

import activation_sparse_gemm_amd as lynx
import tests.gpu_util as gu
from oracle import block_oracle as bo
from tests.gpu_util import host_f64, say
from tests.test_gpu_fp8 import u8
from tests.test_gpu_norm import bf

pytestmark = pytest.mark.gpu

FP8, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu

# every product kernel: few rows; split-K tiles from 32x32 to 128x128; persistent 128x128,
# 256x192 and 256x256 tiles, the first two with even and odd numbers of blocks, each with whole
# and cut pieces of rows; whole and half last blocks of K
SIZES = [(6, 256, 40), (5, 320, 40), (40, 256, 136), (33, 192, 70), (200, 320, 2000), (100, 4160, 3000),
         (300, 320, 3003), (333, 576, 3004), (500, 448, 3000), (190, 192, 9104), (200, 704, 9101), (300, 2176, 9100),
         (350, 2112, 9001), (20, 192, 40001), (50, 192, 40002), (2100, 512, 1552), (2100, 512, 1551), (2100, 640, 1552),
         (2100, 640, 1551), (4608, 256, 4104), (4608, 256, 4101), (4608, 320, 4104), (4608, 320, 4101),
         (9216, 192, 3079), (9216, 256, 3080)]
# scale bytes of X and W, and the power of two that their product stands for
SCALES = [(0, 254, 0), (254, 0, 0), (127, 127, 0), (20, 200, -34), (200, 150, 96), (10, 130, -114),
          (254, 254, "inf"), (254, 240, "inf"), (0, 0, "zero"), (0, 10, "zero")]


@pytest.mark.parametrize("M,K,N", SIZES)
def test_product_of_extreme_scales(M, K, N):
    x = torch.full((M, K), 0x38, dtype=torch.uint8, device="cuda")          # 1.0
    w = torch.full((N, K), 0x38, dtype=torch.uint8, device="cuda").view(FP8)
    x[M // 2] = 0xB8                                                        # a row of -1.0
    x = x.view(FP8)
    words = (K + 511) // 512
    sign = torch.ones((M, 1), device="cuda")
    sign[M // 2] = -1
    for sx, sw, power in SCALES:
        xs = torch.full((words, M, 4), sx, dtype=torch.uint8, device="cuda").view(E8M0)
        ws = torch.full(((N + 127) // 128, 4 * words), sw, dtype=torch.uint8, device="cuda").view(E8M0)
        say(f"extreme scales {sx} {sw} M={M} K={K} N={N}")
        Y = lynx.linear_fp8_packed(x, xs, w, ws, Y=gu.nan_bf16((M, N))).float()
        want = {"inf": float("inf"), "zero": 0.0}.get(power)
        if want is None:
            # K 2^power, one rounding to bf16
            want = torch.tensor(float(K) * 2.0 ** power).to(torch.bfloat16).float().item()
        assert bool((Y == sign * want).all()), (sx, sw, Y[0, 0].item(), Y[M // 2, N - 1].item(), want)


@pytest.mark.parametrize("f32,C", [(False, 640), (True, 640), (True, 2560)])
def test_norm_to_8_bits_at_the_smallest_scale(f32, C):
    """h below 448 2^-127 has the scale 2^-127 and goes down to fp32's subnormals.

    Tolerance: 2^-17 |h| for the arithmetic (no term cancels), an fp32 subnormal's
    rounding 2^-150 in each of two products, and half a step of e4m3: 2^-4 |h|, or
    2^-10 2^-127 for its subnormals."""
    M = 9
    rng = np.random.default_rng(3)
    x = rng.choice([-1.0, 1.0], (M, C)) * np.exp2(rng.uniform(-2, 2, (M, C)))
    X, xf = (torch.from_numpy(x.astype(np.float32)).cuda(), x.astype(np.float32).astype(np.float64)) if f32 else bf(x)
    w = np.ones(C)
    w[:128] = 2.0 ** -122          # the scale's normal range
    w[128:256] = 2.0 ** -130       # its subnormals, and fp32's
    w[256:384] = 2.0 ** -119       # around 448 2^-127
    W, wf = bf(w)
    say(f"smallest scale f32={f32} C={C}")
    q, s = lynx.norm_modulate(X, "rms", weight=W, fp8=True)
    torch.cuda.synchronize()
    _, _, h, _ = bo.block_norm(xf, norm="rms", weight=wf)
    kb = C // 128
    byte = u8(s).transpose(1, 0, 2).reshape(M, -1)[:, :kb]
    want = bo.quantize(h)[1]
    assert (byte[:, :2] == 0).all() and np.array_equal(byte, want)
    v = bo.values(u8(q), byte)
    sub = np.exp2(byte.astype(float) - 127 - 10).repeat(128, 1)
    tol = np.maximum(2.0 ** -4 * np.abs(h), sub) + 2.0 ** -17 * np.abs(h) + 2.0 ** -149
    assert (np.abs(v - h) <= tol).all()
    # the same values as bf16: half a step, or 2^-134 for its subnormals
    hb = host_f64(lynx.norm_modulate(X, "rms", weight=W))
    tol = np.maximum(2.0 ** -8 * np.abs(h), 2.0 ** -134) + 2.0 ** -17 * np.abs(h) + 2.0 ** -149
    assert (np.abs(hb - h) <= tol).all()
