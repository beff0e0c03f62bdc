"""lynx_attention at the ends of fp32: scores far past 2^24, and sums over very many keys."""
import numpy as np
import pytest
import torch

import activation_sparse_gemm_amd as lynx
from tests.gpu_util import host_f64, say
from tests.test_gpu_attention import offsets, randn

pytestmark = pytest.mark.gpu


def far_case(lq, lk, heads, D, seed):
    """q has one channel that is not zero, a power of two that differs from row to row, so scores
    (scale 1) are exact: the key's bf16 number times that power.  Where they are far apart the
    formula gives the mean of the values of the row's largest keys."""
    powers = [0, 2, 24, 27, 33, 40, 60, 100]
    q = torch.zeros((lq, heads, D), dtype=torch.bfloat16, device="cuda")
    e = (torch.arange(lq, device="cuda")[:, None] + 3 * torch.arange(heads, device="cuda")) % len(powers)
    q[..., 0] = torch.tensor([2.0 ** p for p in powers], dtype=torch.bfloat16, device="cuda")[e]
    k, v = randn((lk, heads, D), seed, 2.0), randn((lk, heads, D), seed + 1)
    return q, k, v, np.array(powers)[e.cpu().numpy()]


@pytest.mark.parametrize("lq,lk,heads,D,lens", [
    (130, 300, 2, 64, None), (3, 4000, 2, 128, None), (40, 700, 1, 72, None), (300, 20000, 16, 128, None),
    (4096, 4096, 16, 128, None), (4100, 300, 16, 64, None), (8, 900, 2, 64, [1] * 8),
])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_far_past_2_to_the_24(lq, lk, heads, D, lens, causal, sign):
    q, k, v, powers = far_case(lq, lk, heads, D, 5)
    q = q * sign
    kw = {}
    start, count = np.zeros(lq, dtype=int), np.full(lq, lk)
    if lens:
        lens_k = [lk // len(lens)] * (len(lens) - 1) + [lk - lk // len(lens) * (len(lens) - 1)]
        kw = dict(cu_q=offsets(lens), cu_k=offsets(lens_k))
        start, count = np.cumsum([0] + lens_k[:-1]), np.array(lens_k)
    elif causal:
        count = np.arange(lq) + lk - lq + 1
    say(f"far scores {lq} {lk} {heads}x{D} causal={causal} {sign}")
    out, lse = lynx.attention(q, k, v, causal=causal, scale=1.0, return_lse=True, **kw)
    got, gl = host_f64(out), lse.cpu().numpy().astype(np.float64)
    kn, vn = sign * host_f64(k[..., 0]), host_f64(v)
    rows = np.arange(lq) if lq <= 130 else np.array(sorted({*range(0, lq, 97), *range(24), *range(lq - 24, lq)}))
    none = count[rows] <= 0
    assert (got[rows[none]] == 0).all() and np.isneginf(gl[rows[none]]).all()
    rows = rows[~none]
    key = np.arange(kn.shape[0])[None]
    see = (key >= start[rows, None]) & (key < (start + count)[rows, None])
    n = count[rows]
    for h in range(heads):
        s = np.where(see, kn[None, :, h] * 2.0 ** powers[rows, h][:, None], -np.inf)
        top = s.max(axis=1)
        p = np.exp(s - top[:, None])
        l = p.sum(axis=1)
        want = p @ vn[:, h] / l[:, None]
        dev = np.sqrt(np.maximum(p @ vn[:, h] ** 2 / l[:, None] - want ** 2, 0))
        # products with the factor log2(e) in fp32: 2^-22 of a score that is below 2^6 (the weights of
        # others are 0); scores past that differ by 2^(24 - 7) and more or not at all
        err = n * 2.0 ** -23 + 2.0 ** -21 + np.where(powers[rows, h] < 24, 2.0 ** -22 * 64, 0)
        tol = (2.0 ** -8 + 2 * err)[:, None] * (dev + np.abs(want)) + 1e-30
        assert (np.abs(got[rows, h] - want) <= tol).all()
        # lse = top + log l: log2(e), the product with it, ln 2 and the product with that, 2^-24 each
        assert (np.abs(gl[rows, h] - (top + np.log(l))) <=
                2.0 ** -22 * np.abs(top) + err + 2.0 ** -22 * np.abs(np.log(l))).all()
