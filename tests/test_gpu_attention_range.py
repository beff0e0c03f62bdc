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


@pytest.mark.parametrize("lq,lk,heads", [(130, 300, 2), (3, 4000, 2), (4100, 300, 16), (2048, 2048, 16)])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("power", [24, 28, 29, 30])
def test_scores_on_both_sides_of_a_power_of_two(lq, lk, heads, sign, power):
    """Scores, exact in fp32, that are next to sign * 2^power once they are times log2(e), the first 200 keys'
    a little further down than the others': e^-d of each other, d whole numbers times a score's last place."""
    D = 64
    big = int(2.0 ** power / 1.4426950408889634)
    last = max(1, 2 ** (power - 24))                # a score's last place
    big = big // last * last
    step = last if power < 29 else 4 * last
    pieces, left = [], big
    for _ in range(3):                              # bf16 numbers that add up to it
        unit = 2 ** max(0, left.bit_length() - 8)
        pieces.append(left // unit * unit)
        left -= pieces[-1]
    assert left == 0 and sum(pieces) == big
    rng = np.random.default_rng(power)
    d = rng.integers(-4, 5, lk)
    d[:200] = rng.integers(1, 5, 200)               # first those of small weight
    d[-3:] = -3
    q = torch.zeros((lq, heads, D), dtype=torch.bfloat16, device="cuda")
    q[..., :4] = 1
    k = torch.zeros((lk, heads, D), dtype=torch.bfloat16, device="cuda")
    for i, p in enumerate(pieces):
        k[..., i] = sign * p
    k[..., 3] = torch.from_numpy(-d * step).to(torch.bfloat16).cuda()[:, None]
    v = randn((lk, heads, D), 3)
    say(f"around 2^{power} {lq} {lk} {sign}")
    out, lse = lynx.attention(q, k, v, scale=1.0, return_lse=True)
    p = np.exp(-(d - d.min()).astype(np.float64) * step)
    vn = host_f64(v)
    l = p.sum()
    want = np.einsum("j,jhd->hd", p, vn) / l
    dev = np.sqrt(np.maximum(np.einsum("j,jhd->hd", p, vn ** 2) / l - want ** 2, 0))
    # the factor log2(e) is off by 2^-24 of a difference of 8 steps at most; p and out are rounded.  (Past 2^29
    # the product is off by half its last place, 32 or 64 at most where a step is 128 or 256: the weights of keys
    # that are a step down are 0 either way, and alike keys have alike weights.)
    err = 8 * step * 2.0 ** -23 + 2.0 ** -20 + lk * 2.0 ** -23
    tol = (2.0 ** -8 + 2 * err) * (dev + np.abs(want)) + 1e-30
    got = host_f64(out)
    assert (np.abs(got - want[None]) <= tol[None]).all()
    top = sign * float(big) - d.min() * step
    gl = lse.cpu().numpy().astype(np.float64)
    assert (np.abs(gl - (top + np.log(l))) <= 2.0 ** -22 * abs(top) + 1e-3).all()


@pytest.mark.parametrize("name", ["256-row tiles", "128-row tiles", "few rows"])
def test_sums_over_very_many_keys(name):
    """Keys that are all alike: every weight is the same number, so that additions to a growing sum
    all round the same way.  lse's bound does not grow with the number of keys: a score's error, a tile's
    sum (2^-20 with the power of two and the logarithm), lse's own rounding.  out's sums are
    rounded every 16 keys, its divisor's every tile: n / 16 2^-24 each at most."""
    D, heads, seqs, lq, lk = {"256-row tiles": (8, 16, 1, 8192, 262144), "128-row tiles": (8, 16, 2, 4096, 131072),
                              "few rows": (64, 1, 512, 1, 131072)}[name]
    q, k = randn((seqs * lq, heads, D), 1), randn((1, heads, D), 2)
    v = torch.full((1, heads, D), 1.25, dtype=torch.bfloat16, device="cuda")
    say(f"sums over many keys, {name}")
    if name == "few rows":  # all sequences share one cache
        K, V = (t.expand(lk, heads, D).contiguous().unsqueeze(0).expand(seqs, lk, heads, D) for t in (k, v))
        out, lse = lynx.attention(q.view(seqs, lq, heads, D), K, V, return_lse=True)
    else:
        K, V = (t.expand(seqs * lk, heads, D).contiguous() for t in (k, v))
        cu = (offsets([lq] * seqs), offsets([lk] * seqs)) if seqs > 1 else (None, None)
        out, lse = lynx.attention(q, K, V, *cu, return_lse=True)
    qd, kd = q.double(), k.double()
    s, spread = (qd * kd).sum(-1) * D ** -0.5, (qd * kd).abs().sum(-1) * D ** -0.5
    want = s + np.log(lk)
    tol = (D * 2.0 ** -23 + 2.0 ** -22) * spread + 2.0 ** -21 + 2.0 ** -20 + 2.0 ** -22 * want.abs()
    err = (lse.double().reshape(want.shape) - want).abs()
    say(f"lse off by {err.max().item():.2e}, {(err / tol).max().item():.3f} of its bound")
    assert (err <= tol).all()
    assert ((out.double() - 1.25).abs() <= 1.25 * (2.0 ** -8 + 2 * lk / 16 * 2.0 ** -24)).all()
