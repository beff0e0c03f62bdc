"""lynx_qk_rotary against the fp64 oracle.

Tolerance per element: one rounding to bf16, 2^-8 relative; before it fp32 products and sums
and a cosine and sine of an angle that is within 2^-24 of a turn (2 pi 2^-24 < 2^-21), with
the functions' own error below 2^-22: 2^-20 of the pair's size.  With a norm the factor
rsqrt(mean square + eps) has relative error (D + 4) 2^-24 at most.
"""
import numpy as np
import pytest
import torch

import activation_sparse_gemm_amd as lynx
from oracle import attention_oracle as ao
from tests.gpu_util import host_f64, nan_bf16, say
from tests.test_gpu_attention import randn

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def pair_size(x, axes, pairs):
    """The norm of each channel's pair (the channel itself where it is not turned)."""
    R = sum(axes)
    s = np.abs(x)
    c = np.arange(R)
    other = c ^ 1 if pairs == "adjacent" else (c + R // 2) % R
    s[..., :R] = np.hypot(x[..., :R], x[..., other])
    return s


def check(got, x, positions, axes, theta, pairs, ladder, norm=False, weight=None, eps=1e-6):
    pos = positions.cpu().numpy()
    kw = dict(norm=norm, weight=None if weight is None else host_f64(weight), eps=eps)
    ref = ao.rotary(host_f64(x), pos, axes, theta, pairs, ladder, **kw)
    flat = ao.rotary(host_f64(x), np.zeros_like(pos), axes, theta, pairs, ladder, **kw)
    D = x.shape[-1]
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -20 + (D + 4) * 2.0 ** -24) * pair_size(flat, axes, pairs) + 1e-30
    err = np.abs(host_f64(got) - ref)
    say(f"worst {np.max(err / tol):.3f} of its bound")
    assert (err <= tol).all(), f"{(err > tol).sum()} outside, first {np.argwhere(err > tol)[0]}"


def positions_of(T, n, f32, seed, far=1000):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    p = torch.randint(-far, far, (T, n), device="cuda", generator=g, dtype=torch.int32)
    return p.float() * 0.37 if f32 else p


def run(T, H, KV, D, axes, theta=1e4, pairs="adjacent", ladder="axis", norm=False, weights=False, f32=False,
        far=1000, seed=1):
    q, k = randn((T, H, D), seed, 3.0), randn((T, KV, D), seed + 1) if KV else None
    pos = positions_of(T, len(axes), f32, seed + 2, far)
    qw, kw = (randn((D,), seed + 3), randn((D,), seed + 4) if KV else None) if weights else (None, None)
    out = nan_bf16((T, H, D)), nan_bf16((T, KV, D)) if KV else None
    say(f"rotary {T}x{H}+{KV}x{D} {axes} {pairs} {ladder} norm={norm} f32={f32}")
    qo, ko = lynx.qk_rotary(q, k, pos, axes, theta, pairs, ladder, "rms" if norm else None, qw, kw, out=out)
    torch.cuda.synchronize()
    check(qo, q, pos, axes, theta, pairs, ladder, norm, qw)
    if KV:
        check(ko, k, pos, axes, theta, pairs, ladder, norm, kw)


@pytest.mark.parametrize("D,axes", [
    (8, (2,)), (8, (8,)), (32, (2, 4, 6)), (40, (18, 20)), (64, (64,)), (64, (30, 30)), (64, (16, 24, 24)),
    (72, (16, 24, 24)), (80, (80,)), (96, (2, 2, 2, 90)), (104, (50, 54)), (128, (16, 56, 56)), (128, (128,)),
    (128, (32, 32)), (136, (34, 34, 34, 34)), (192, (64, 64, 64)), (256, (256,)), (256, (6, 8)),
])
@pytest.mark.parametrize("pairs", ["adjacent", "halves"])
@pytest.mark.parametrize("ladder", ["axis", "joint"])
def test_head_sizes_and_axes(D, axes, pairs, ladder):
    run(7, 3, 2, D, axes, pairs=pairs, ladder=ladder)
    run(7, 3, 2, D, axes, pairs=pairs, ladder=ladder, norm=True, weights=True, f32=True)


@pytest.mark.parametrize("D", list(range(8, 257, 8)))
@pytest.mark.parametrize("pairs", ["adjacent", "halves"])
def test_norm_of_every_head_size(D, pairs):
    run(5, 9, 2, D, (D // 4 * 2, D // 4 * 2), pairs=pairs, norm=True, weights=True)


@pytest.mark.parametrize("T,H,KV", [
    (1, 1, 0), (1, 40, 8), (2, 1, 1), (1000, 1, 0), (333, 5, 1), (17, 24, 24), (4100, 3, 3), (3, 1024, 1024),
])
@pytest.mark.parametrize("pairs", ["adjacent", "halves"])
@pytest.mark.parametrize("norm", [False, True])
def test_tokens_and_heads(T, H, KV, pairs, norm):
    run(T, H, KV, 64, (16, 24, 24), pairs=pairs, norm=norm)


@pytest.mark.parametrize("theta", [2.0, 256.0, 1e6])
@pytest.mark.parametrize("f32", [False, True])
def test_far_positions(theta, f32):
    """Angles of millions of turns keep their fraction."""
    run(50, 2, 1, 128, (64, 64), theta=theta, far=2 ** 30, f32=f32, ladder="joint")
    run(50, 2, 1, 128, (128,), theta=theta, far=2 ** 24, f32=f32, pairs="halves")


@pytest.mark.parametrize("theta,axes", [(1.5, (256,)), (2.0, (128, 128)), (2.0, (128,)), (1e4, (128,))])
@pytest.mark.parametrize("ladder", ["axis", "joint"])
def test_angles_at_the_last_positions(theta, axes, ladder):
    """Positions next to 2^31, and channels that nearly cancel, so that the result's own rounding hides
    nothing.  An angle's frequency and the angle are rounded to 53 bits, 2^-52 of the angle together;
    what is left of whole turns is rounded to fp32, half a turn at most: 2 pi 2^-26 < 2^-23.3; cosine and
    sine are off by 2^-23 each, the products by 2^-24: (2^-52 angle + 2^-21.4) of the pair's size."""
    LD = np.longdouble
    T, R = 64, sum(axes)
    g = np.random.default_rng(3)
    pos = np.stack([2 ** 31 - 1 - g.integers(0, 1 << 20, T) for _ in axes], 1)
    pos[::2] *= -1
    angle, p = np.zeros((T, R // 2), dtype=LD), 0
    for i, d in enumerate(axes):
        for j in range(d // 2):
            e = LD(j) / LD(d // 2) if ladder == "axis" else LD(p) / LD(R // 2)
            angle[:, p] = pos[:, i].astype(LD) * LD(theta) ** -e
            p += 1
    c, s = np.cos(angle), np.sin(angle)

    def bf16(x):
        return torch.from_numpy(np.asarray(x, dtype=np.float64)).to(torch.bfloat16).double().numpy()

    # x_m c = x_n s nearly: the larger of the two one of 128 numbers in [1, 2), the other rounded
    lead = (1 + np.arange(128) / 128)[None, None].astype(LD)
    big_m = np.abs(s) >= np.abs(c)
    ratio = np.where(big_m, c / np.where(s == 0, 1, s), s / np.where(c == 0, 1, c))[..., None]
    small = bf16(lead * ratio)
    m = np.where(big_m[..., None], lead, small)
    n = np.where(big_m[..., None], small, lead)
    best = np.abs(m * c[..., None] - n * s[..., None]).argmin(-1)[..., None]
    m, n = (np.take_along_axis(np.broadcast_to(t, m.shape), best, -1)[..., 0] for t in (m, n))
    x = torch.zeros((T, 1, R), dtype=torch.bfloat16)
    x[:, 0, 0::2], x[:, 0, 1::2] = torch.from_numpy(m.astype(np.float64)), torch.from_numpy(n.astype(np.float64))
    say(f"last positions {theta} {axes} {ladder}")
    got, _ = lynx.qk_rotary(x.cuda(), None, torch.from_numpy(pos.astype(np.int32)).cuda(), axes, theta,
                            ladder=ladder)
    want = (m * c - n * s).astype(np.float64)
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -52 * np.abs(angle) + 2.0 ** -21.4).astype(np.float64) * np.hypot(m, n)
    err = np.abs(host_f64(got)[:, 0, 0::2] - want)
    say(f"worst {np.max(err / tol):.3f} of its bound")
    assert (err <= tol.astype(np.float64)).all()


@pytest.mark.parametrize("pairs", ["adjacent", "halves"])
def test_slices_of_a_projection_in_place(pairs):
    T, H, KV, D = 77, 6, 2, 72
    qkv = randn((T, H + 2 * KV, D), 1)
    pos = positions_of(T, 3, False, 2)
    q, k = qkv[:, :H], qkv[:, H:H + KV]
    q0, k0, v0 = q.clone(), k.clone(), qkv[:, H + KV:].clone()
    say("in place")
    got = lynx.qk_rotary(q, k, pos, (24, 24, 24), pairs=pairs, norm="rms", out=(q, k))
    assert got[0] is q and got[1] is k
    check(q, q0, pos, (24, 24, 24), 1e4, pairs, "axis", True)
    check(k, k0, pos, (24, 24, 24), 1e4, pairs, "axis", True)
    assert torch.equal(qkv[:, H + KV:], v0)
    # heads before tokens
    x = randn((H, T, D), 3).transpose(0, 1)
    o = nan_bf16((H, T, D)).transpose(0, 1)
    lynx.qk_rotary(x, None, pos, (24, 24, 24), pairs=pairs, out=(o, None))
    check(o, x, pos, (24, 24, 24), 1e4, pairs, "axis")


@pytest.mark.parametrize("pairs", ["adjacent", "halves"])
def test_negated_positions_undo_the_turn(pairs):
    """The gradient of a turn: <turn(x), y> = <x, turn back(y)> up to bf16's rounding."""
    x, y = randn((60, 4, 64), 1), randn((60, 4, 64), 2)
    pos = positions_of(60, 3, False, 3)
    a = host_f64(lynx.qk_rotary(x, None, pos, (16, 24, 24), pairs=pairs)[0])
    b = host_f64(lynx.qk_rotary(y, None, -pos, (16, 24, 24), pairs=pairs)[0])
    x, y = host_f64(x), host_f64(y)
    lhs, rhs = (a * y).sum(-1), (x * b).sum(-1)
    bound = (2.0 ** -8 + 2.0 ** -18) * (np.abs(a) * np.abs(y) + np.abs(x) * np.abs(b)).sum(-1)
    assert (np.abs(lhs - rhs) <= bound * (1 + 2.0 ** -7)).all()


@pytest.mark.parametrize("pairs", ["adjacent", "halves"])
@pytest.mark.parametrize("norm", [None, "rms"])
def test_values_that_are_not_finite(pairs, norm):
    T, H, D, axes = 9, 3, 64, (16, 24)
    x, pos = randn((T, H, D), 1), positions_of(T, 2, True, 2)
    want, _ = lynx.qk_rotary(x, None, pos, axes, pairs=pairs, norm=norm)
    x[1, 0, 3], x[2, 1, 63], x[4, 2, 20] = INF, NAN, 3e38
    pos[6, 1] = NAN
    say(f"not finite {pairs} {norm}")
    got, _ = lynx.qk_rotary(x, None, pos, axes, pairs=pairs, norm=norm)
    bad = torch.zeros((T, H, D), dtype=torch.bool, device="cuda")
    i = torch.arange(40, device="cuda")
    pair = i // 2 if pairs == "adjacent" else i % 20
    bad[6, :, :40] = pair >= 8                     # the second axis' pairs
    if norm:
        bad[1, 0] = bad[2, 1] = bad[4, 2] = True
        assert torch.isnan(got[bad]).all()
    else:
        for t, h, c in ((1, 0, 3), (4, 2, 20)):    # (3e38 may stay finite)
            bad[t, h, :40] |= pair == pair[c]
        bad[2, 1, 63] = True
        assert torch.isnan(got[2, 1, 63]) and not torch.isfinite(got[1, 0][bad[1, 0]]).any()
        assert torch.isnan(got[6][bad[6]]).all()
    assert torch.equal(got[~bad], want[~bad])


def test_outputs_go_with_inputs():
    x, pos = randn((3, 2, 64), 1), positions_of(3, 1, False, 2)
    for k, out in ((x, (x, None)), (None, (x, x))):
        with pytest.raises(ValueError, match="second output"):
            lynx.qk_rotary(x, k, pos, (64,), out=out)


def test_a_norm_of_zeros_and_of_small_rows():
    x = randn((4, 2, 64), 1)
    x[0] = 0
    x[1] *= 2.0 ** -60
    pos = positions_of(4, 1, False, 2)
    got, _ = lynx.qk_rotary(x, None, pos, (64,), norm="rms")
    check(got, x, pos, (64,), 1e4, "adjacent", "axis", True)
    assert (got[0] == 0).all()


def test_rows_past_32_bits():
    """Tokens far apart in memory: element offsets past 2^31."""
    T, stride = 5, 1 << 30
    base = torch.zeros(((T - 1) * stride + 128,), dtype=torch.bfloat16, device="cuda")
    x = base.as_strided((T, 2, 64), (stride, 64, 1))
    x.copy_(randn((T, 2, 64), 1))
    x0, pos = x.clone(), positions_of(T, 1, False, 2)
    say("far rows")
    lynx.qk_rotary(x, None, pos, (64,), out=(x, None))
    check(x, x0, pos, (64,), 1e4, "adjacent", "axis")


def test_captured_and_replayed():
    q, k, pos = randn((300, 4, 128), 1), randn((300, 2, 128), 2), positions_of(300, 3, False, 3)
    out = nan_bf16((300, 4, 128)), nan_bf16((300, 2, 128))
    args = (q, k, pos, (16, 56, 56))
    ref = [t.clone() for t in lynx.qk_rotary(*args, norm="rms")]
    lynx.qk_rotary(*args, norm="rms", out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lynx.qk_rotary(*args, norm="rms", out=out)
    for _ in range(3):
        for o in out:
            o.view(torch.int16).fill_(0x7FC0)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, ref))
    pos.neg_()
    g.replay()
    want = lynx.qk_rotary(*args, norm="rms")
    assert all(torch.equal(a, b) for a, b in zip(out, want))


# ---- with attention ---------------------------------------------------------------

def test_the_attention_half_of_a_block():
    """norm -> QKV -> qk_rotary -> attention -> output projection -> residual, through the library
    alone, against the same in 64 bits from each stage's own input (bf16 between stages)."""
    from oracle import block_oracle as bo
    T, H, D, C = [200, 57], 4, 64, 256
    n = sum(T)
    x, W, Wo = randn((n, C), 1), randn((3 * C, C), 2, C ** -0.5), randn((C, C), 3, C ** -0.5)
    scale, shift, gate = (randn((2, C), s, 0.3) for s in (4, 5, 6))
    qw, kw = randn((D,), 7, 0.2) + 1, randn((D,), 8, 0.2) + 1
    pos = torch.stack([torch.arange(n, device="cuda") // 16, torch.arange(n, device="cuda") % 16], 1).int()
    cu = torch.tensor([0, 200, 257], dtype=torch.int32, device="cuda")
    say("block half")
    h = lynx.norm_modulate(x, "layer", scale=scale[:1], shift=shift[:1])
    qkv = lynx.linear_dense(h, W).view(n, 3 * H, D)
    q, k = lynx.qk_rotary(qkv[:, :H], qkv[:, H:2 * H], pos, (32, 32), norm="rms", q_weight=qw, k_weight=kw)
    a = lynx.attention(q, k, qkv[:, 2 * H:], cu)
    y = lynx.linear_dense(a.view(n, C), Wo)
    x2, _ = lynx.residual_norm(x, y, gate=gate[:1])
    q64 = ao.rotary(host_f64(qkv[:, :H]), pos.cpu().numpy(), (32, 32), norm=True, weight=host_f64(qw))
    k64 = ao.rotary(host_f64(qkv[:, H:2 * H]), pos.cpu().numpy(), (32, 32), norm=True, weight=host_f64(kw))
    check(q, qkv[:, :H], pos, (32, 32), 1e4, "adjacent", "axis", True, qw)
    check(k, qkv[:, H:2 * H], pos, (32, 32), 1e4, "adjacent", "axis", True, kw)
    a64 = ao.attention(q64, k64, host_f64(qkv[:, 2 * H:]), T, T)[0].reshape(n, C)
    y64 = a64 @ host_f64(Wo).T
    x64 = host_f64(x) + host_f64(gate[:1]) * y64
    # q, k, the weights, a, y and x' are rounded: each at most 2^-8 of its size, q and k by way of
    # the scores, which reach about 8: 2 * 8 * 2^-8 of a's size at most, so 5e-2 in all; x' once more
    err = np.linalg.norm(host_f64(x2) - x64, axis=1) / np.linalg.norm(x64, axis=1)
    say(f"block half: worst row {err.max():.2e}")
    assert err.max() <= 5e-2
    assert bo is not None


def test_the_stages_before_the_turn():
    """norm -> QKV, each against 64 bits of its own input (the block's half above starts at their result).

    h: rounded once, 2^-8; before it mean, variance, their factor and the shift in fp32: sums of C terms
    in trees and chains of less than 2^6, so 2^-17 of the magnitudes that are added.  qkv: rounded once, and
    C products summed in fp32, C 2^-24 of their magnitudes."""
    n, C = 257, 256
    x, W = randn((n, C), 1), randn((3 * C, C), 2, C ** -0.5)
    scale, shift = randn((1, C), 4, 0.3), randn((1, C), 5, 0.3)
    say("norm and projection before the turn")
    h = lynx.norm_modulate(x, "layer", scale=scale, shift=shift)
    qkv = lynx.linear_dense(h, W)
    X = host_f64(x)
    t = X - X.mean(1, keepdims=True)
    f = (1 + host_f64(scale)) / np.sqrt((t * t).mean(1, keepdims=True) + 1e-6)
    want = t * f + host_f64(shift)
    mag = (np.abs(X) + np.abs(X).mean(1, keepdims=True)) * np.abs(f) + np.abs(host_f64(shift))
    assert (np.abs(host_f64(h) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -17 * mag).all()
    H, Wn = host_f64(h), host_f64(W)
    want = H @ Wn.T
    assert (np.abs(host_f64(qkv) - want) <= 2.0 ** -8 * np.abs(want) + C * 2.0 ** -24 * (np.abs(H) @ np.abs(Wn).T)).all()
