"""lynx_attention against the fp64 oracle.

Tolerances, per element.  The library rounds p to bf16 for the product and the sum alike,
d_j relative, |d_j| <= 2^-8: out is then off by sum p_j d_j (v_j - out) / sum p_j, at most
2^-8 sum p |v - out| / sum p <= 2^-8 dev (dev: the weighted standard deviation).  out is
rounded once: 2^-8 |out|.  A score is a sum of D products in fp32, off by D 2^-23 times the sum
of magnitudes at most, then there are a fused multiply-add and a power of two (2^-21
together, and 2^-22 of the score); numerator and denominator change by that, and sums of n
terms in fp32 by n 2^-24 of their magnitudes (sum p |v| <= sum p |v - out| + |out| sum p).
lse: the score's error, the sum's and its own rounding.

And per row, against mistakes that such bounds let pass, the library's bar of 5e-3:
of |out| for its rounding (2^-8 at most), and of `size` for the d_j: independent, rms
2^-8 / sqrt(3) at most, they give an error of 2.3e-3 size, and with 8 channels or more twice
that is ten standard deviations off.
"""
import numpy as np
import pytest
import torch

import activation_sparse_gemm_amd as lynx
from oracle import attention_oracle as ao
from tests.gpu_util import host_f64, nan_bf16, poisoned_bytes, say

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def randn(shape, seed, size=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (size * torch.randn(shape, device="cuda", generator=g)).to(torch.bfloat16)


def offsets(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def check(out, lse, ref, D, n):
    """out, lse of the library (device) against ao.attention's results; n: keys of the longest
    sequence, prefix included."""
    o, l, dev, size, spread = ref
    got = host_f64(out).reshape(o.shape)
    err_s = D * 2.0 ** -23 * spread + 2.0 ** -22 * spread + 2.0 ** -21
    tol = 2.0 ** -8 * (dev + np.abs(o)) + (2 * err_s[..., None] + n * 2.0 ** -23) * (dev + np.abs(o)) + 1e-30
    bad = ~(np.abs(got - o) <= tol)
    assert not bad.any(), f"{bad.sum()} outside, first {np.argwhere(bad)[0]}, " \
        f"off by {np.abs(got - o)[bad][:3]} of {tol[bad][:3]}"
    empty = np.isneginf(l)
    assert (got[empty] == 0).all()
    err = np.linalg.norm(got - o, axis=-1) / np.maximum(np.linalg.norm(o, axis=-1) + size, 1e-30)
    say(f"worst row {err.max():.2e}, mean {err.mean():.2e}, worst of its bound {(np.abs(got - o) / tol).max():.2f}")
    assert err.max() <= 5e-3
    if lse is not None:
        gl = lse.cpu().numpy().astype(np.float64).reshape(l.shape)
        assert np.isneginf(gl[empty]).all()
        tl = err_s + n * 2.0 ** -23 + 2.0 ** -22 * np.abs(l)
        assert (np.abs(gl[~empty] - l[~empty]) <= tl[~empty]).all()


def poisoned(q, B, Tk, kv, P, packed, causal):
    """out, lse and workspace that hold what no call may read or leave."""
    Tq = q.numel() // (q.shape[-1] * q.shape[-2])
    n = lynx.attention_workspace_bytes(B, Tq, Tk, q.shape[-2], kv, q.shape[-1], P, packed, causal)
    return dict(out=nan_bf16(tuple(q.shape)),
                lse=torch.full(q.shape[:-1], NAN, device="cuda"), workspace=poisoned_bytes(n))


def packed_case(lens_q, lens_k, heads, kv, D, causal, seed, P=0, scale=None, size=1.6):
    q, k, v = randn((sum(lens_q), heads, D), seed, size), randn((sum(lens_k), kv, D), seed + 1, size), \
        randn((sum(lens_k), kv, D), seed + 2)
    prefix = (randn((P, kv, D), seed + 3, size), randn((P, kv, D), seed + 4)) if P else None
    ref = ao.attention(host_f64(q), host_f64(k), host_f64(v), lens_q, lens_k, causal, scale,
                       tuple(map(host_f64, prefix)) if P else None)
    say(f"packed q={lens_q[:8]} k={lens_k[:8]} n={len(lens_q)} {heads}/{kv}x{D} causal={causal} P={P}")
    out, lse = lynx.attention(q, k, v, offsets(lens_q), offsets(lens_k), causal, scale, prefix,
                              **poisoned(q, len(lens_q), sum(lens_k), kv, P, True, causal))
    torch.cuda.synchronize()
    check(out, lse, ref, D, max(lens_k) + P)
    return out, lse


EDGES = [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 257]


@pytest.mark.parametrize("D", [8, 24, 32, 40, 64, 72, 80, 96, 104, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_head_sizes(D, causal):
    packed_case([130, 65], [130, 65], 2, 2, D, causal, 10 + D)
    packed_case([1, 3], [130, 65], 4, 2, D, causal, 11 + D)


@pytest.mark.parametrize("heads,kv", [(1, 1), (3, 1), (4, 2), (8, 8), (12, 12), (14, 2), (10, 5), (40, 1)])
@pytest.mark.parametrize("causal", [False, True])
def test_grouped_heads(heads, kv, causal):
    packed_case([70, 1, 9, 200], [70, 50, 300, 200], heads, kv, 64, causal, 20 + heads)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_lengths_at_the_tiles_ends(D, causal):
    packed_case(EDGES, EDGES, 2, 1, D, causal, 30)
    packed_case(EDGES, EDGES[::-1], 2, 2, D, causal, 31)     # Lq > Lk too: rows that see nothing


@pytest.mark.parametrize("causal", [False, True])
def test_empty_sequences(causal):
    packed_case([0, 5, 0, 40, 0], [3, 0, 0, 70, 9], 4, 2, 128, causal, 40)
    packed_case([300, 5, 0], [0, 0, 9], 4, 2, 64, causal, 41)
    packed_case([5], [0], 2, 2, 64, causal, 42)


@pytest.mark.parametrize("lens_q", [1, 2, 7])
@pytest.mark.parametrize("causal", [False, True])
def test_many_sequences(lens_q, causal):
    """More sequences than lanes, caches of very different lengths (one of thousands of keys)."""
    rng = np.random.default_rng(lens_q)
    lk = [int(x) for x in np.exp(rng.uniform(0, 5, 150))]
    lk[17], lk[149] = 5000, 700
    packed_case([lens_q] * 150, [max(n, lens_q) for n in lk], 4, 2, 64, causal, 50 + lens_q)


@pytest.mark.parametrize("n", [2, 63, 64, 65, 130])
@pytest.mark.parametrize("causal", [False, True])
def test_row_tiles_of_many_sequences(n, causal):
    # lengths that rise and fall, some of them alike, some zero
    lens = [(37 * i) % 90 * (i % 5 != 3) + 20 * (i % 7 == 0) for i in range(n)]
    packed_case(lens, [a + (i * 11) % 50 for i, a in enumerate(lens)], 4, 2, 64, causal, 3)
    packed_case(lens, lens, 2, 2, 128, causal, 4, P=65)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_one_long_sequence_among_single_tokens(D, causal):
    # the long one has 38 row tiles of 32, and several chunks of keys
    n = 60
    lens_q, lens_k = [1] * n + [300] + [1] * n, list(range(1, 7 * n, 7)) + [4000] + [33] * n
    packed_case(lens_q, lens_k, 4, 1, D, causal, 5)
    packed_case(lens_q, lens_k, 4, 1, D, causal, 9, P=700)


@pytest.mark.parametrize("lq,lk,heads,kv,D", [
    (1, 1, 1, 1, 128), (1, 9000, 8, 1, 128), (4, 5001, 8, 8, 64), (33, 4100, 1, 1, 128),
    (100, 6000, 2, 2, 128), (200, 3001, 4, 1, 72), (1, 700, 64, 1, 128), (700, 40, 2, 1, 128),
])
@pytest.mark.parametrize("causal", [False, True])
def test_one_sequence(lq, lk, heads, kv, D, causal):
    """Few rows and long keys: keys are cut and joined."""
    packed_case([lq], [lk], heads, kv, D, causal, 60 + lq)


@pytest.mark.parametrize("lens_q,lens_k,P", [
    ([1, 1, 1], [1, 40, 300], 1), ([1] * 40, list(range(1, 41)), 700), ([2, 0, 5], [2, 9, 0], 130),
    ([200, 300], [200, 300], 65), ([9], [20], 1000), ([1], [1], 3000), ([40, 1], [0, 0], 50),
])
@pytest.mark.parametrize("heads,kv,D", [(4, 4, 64), (8, 2, 128), (3, 1, 40)])
@pytest.mark.parametrize("causal", [False, True])
def test_shared_prefix(lens_q, lens_k, P, heads, kv, D, causal):
    packed_case(lens_q, lens_k, heads, kv, D, causal, 70 + P, P)


@pytest.mark.parametrize("lens_q,lens_k,heads,kv,P", [
    ([1, 1], [9, 11], 8, 1, 70000), ([1] * 4, [5, 0, 300, 1], 12, 2, 100000), ([1, 2], [30, 2], 8, 2, 84489),
    ([3, 0, 1], [3, 7, 1], 3, 3, 96488), ([1] * 4, [5, 0, 300, 1], 12, 2, 65536),
])
@pytest.mark.parametrize("D", [64, 128])
def test_a_long_prefix_of_few_key_heads(lens_q, lens_k, heads, kv, P, D):
    """The prefix is cut into the most pieces that there are, or, since pieces are of whole tiles,
    fewer: the join reads no others (the workspace holds NaN)."""
    packed_case(lens_q, lens_k, heads, kv, D, True, 90 + kv, P)


def test_the_prefix_is_the_keys_before():
    """The same keys as a prefix and as each sequence's own give the same result, up to rounding."""
    lens, P = [3, 50, 129], 200
    q, k, v = randn((182, 4, 64), 1), randn((182, 2, 64), 2), randn((182, 2, 64), 3)
    pk, pv = randn((P, 2, 64), 4), randn((P, 2, 64), 5)
    at = np.concatenate([[0], np.cumsum(lens)])

    def own(t, p):
        return torch.cat([torch.cat([p, t[a:b]]) for a, b in zip(at[:-1], at[1:])])

    say("prefix against own keys")
    a, la = lynx.attention(q, k, v, offsets(lens), causal=True, prefix=(pk, pv), return_lse=True)
    b, lb = lynx.attention(q, own(k, pk), own(v, pv), offsets(lens), offsets([n + P for n in lens]),
                           causal=True, return_lse=True)
    assert torch.allclose(la, lb, rtol=0, atol=2e-5)
    assert (a.float() - b.float()).abs().max() <= 2 ** -7 * b.float().abs().max() + 2 ** -7


@pytest.mark.parametrize("B,Lq,Lk,heads,kv,D", [
    (1, 77, 77, 3, 3, 64), (2, 300, 130, 4, 2, 72), (3, 1, 1000, 8, 2, 128), (2, 5, 0, 2, 1, 64),
])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("layout", ["BSHD", "BHSD", "slices"])
def test_uniform_batches_and_strides(B, Lq, Lk, heads, kv, D, causal, layout):
    def make(L, h, seed):
        if layout == "BHSD":
            return randn((B, h, L, D), seed).transpose(1, 2)
        if layout == "slices":
            return randn((B, L, h + 2, D + 8), seed)[:, :, 1:1 + h, 8:]
        return randn((B, L, h, D), seed)

    q, k, v = make(Lq, heads, 1), make(Lk, kv, 2), make(Lk, kv, 3)
    ref = ao.attention(*(host_f64(t).reshape(-1, t.shape[2], D) for t in (q, k, v)), [Lq] * B, [Lk] * B,
                       causal)
    say(f"uniform {layout} {B}x{Lq}x{Lk} {heads}/{kv}x{D} causal={causal}")
    kw = poisoned(q, B, B * Lk, kv, 0, False, causal)
    if layout == "BHSD":
        kw["out"] = nan_bf16((B, heads, Lq, D)).transpose(1, 2)
    out, lse = lynx.attention(q, k, v, causal=causal, **kw)
    check(out, lse, ref, D, Lk)


@pytest.mark.parametrize("B,Lq,Lk,heads,kv,D", [
    (2, 4100, 300, 16, 16, 72), (5, 2011, 1, 16, 4, 128), (3, 3001, 640, 12, 12, 64), (1, 4609, 77, 24, 3, 40),
    (1, 9000, 320, 14, 2, 128), (70, 131, 33, 16, 8, 96), (1, 8200, 65, 32, 8, 128), (300, 260, 64, 2, 2, 8),
])
@pytest.mark.parametrize("layout", ["BSHD", "BHSD"])
def test_many_rows_on_few_keys(B, Lq, Lk, heads, kv, D, layout):
    def make(L, h, seed, size=1.6):
        if layout == "BHSD":
            return randn((B, h, L, D), seed, size).transpose(1, 2)
        return randn((B, L, h + 1, D + 8), seed, size)[:, :, 1:, 8:]

    q, k, v = make(Lq, heads, 1), make(Lk, kv, 2), make(Lk, kv, 3, 1.0)
    some = sorted({0, 1, 31, 32, 33, Lq // 2, Lq - 33, Lq - 32, Lq - 2, Lq - 1})
    ref = ao.attention(host_f64(q[:, some]).reshape(-1, heads, D),
                       *(host_f64(t).reshape(-1, kv, D) for t in (k, v)), [len(some)] * B, [Lk] * B, False)
    say(f"few keys {layout} {B}x{Lq}x{Lk} {heads}/{kv}x{D}")
    kw = poisoned(q, B, B * Lk, kv, 0, False, False)
    if layout == "BHSD":
        kw["out"] = nan_bf16((B, heads, Lq, D)).transpose(1, 2)
    out, lse = lynx.attention(q, k, v, **kw)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    check(out[:, some], lse[:, some], ref, D, Lk)
    # other rows, as a call of few rows, which another kernel takes: twice the bounds above, with
    # dev <= 2 max |v| and magnitudes of a score <= scale |q| |k|
    n = min(500, Lq)
    other, lother = lynx.attention(q[:1, :n], k[:1], v[:1], return_lse=True)
    spread = (q[:1, :n].float().norm(dim=-1).max() * k[:1].float().norm(dim=-1).max()).item() * D ** -0.5
    err_s = (D * 2.0 ** -23 + 2.0 ** -22) * spread + 2.0 ** -21
    top = 3 * v[:1].float().abs().max().item()
    assert (out[0, :n].float() - other[0].float()).abs().max() <= 2 * (2.0 ** -8 + 2 * err_s + Lk * 2.0 ** -23) * top
    assert (lse[0, :n] - lother[0]).abs().max() <= \
        2 * (err_s + Lk * 2.0 ** -23 + 2.0 ** -22 * lother[0].abs().max().item())


def test_heads_may_share_memory():
    q, k = randn((100, 6, 64), 1), randn((100, 1, 64), 2)
    v = randn((100, 1, 64), 3)
    a = lynx.attention(q, k.expand(100, 3, 64), v.expand(100, 3, 64), causal=True)
    ref = ao.attention(host_f64(q), host_f64(k), host_f64(v), [100], [100], True)
    check(a, None, ref, 64, 100)


@pytest.mark.parametrize("scale", [1e-3, 1.0, 30.0])
@pytest.mark.parametrize("lens", [[150], [1] * 5])
def test_scales(scale, lens):
    packed_case(lens, [n + 100 for n in lens], 2, 2, 64, True, 80, scale=scale)


@pytest.mark.parametrize("lq,lk", [(130, 300), (1, 3000)])
def test_scores_that_rise_and_fall(lq, lk):
    """Maxima that grow from key to key by far more than the lead a row keeps, and fall."""
    D = 64
    q = torch.zeros((lq, 1, D), dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 1
    k, v = randn((lk, 1, D), 1), randn((lk, 1, D), 2)
    for shape in (np.linspace(0, 400, lk), np.linspace(300, -300, lk), 200 * np.sin(np.arange(lk) / 40),
                  np.where(np.arange(lk) == lk - 1, 1e4, -1e4)):
        k[:, 0, 0] = torch.from_numpy(shape).to(torch.bfloat16).cuda()
        ref = ao.attention(host_f64(q), host_f64(k), host_f64(v), [lq], [lk], True, 1.0)
        say(f"rising scores {lq} {lk}")
        out, lse = lynx.attention(q, k, v, causal=True, scale=1.0, return_lse=True)
        check(out, lse, ref, D, lk)


# ---- what must have no influence ---------------------------------------------------

def spoiled(t, rows):
    t = t.clone()
    t[rows] = torch.tensor([NAN, INF, -INF, 3e38] * (t.shape[-1] // 4), dtype=torch.bfloat16, device="cuda")
    return t


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens_q,lens_k", [([130, 1, 60], [130, 33, 60]), ([1, 1, 2], [129, 33, 60])])
@pytest.mark.parametrize("D", [40, 64, 128])
def test_rows_outside_of_the_sequences(D, lens_q, lens_k, causal):
    """NaN and infinities around a sequence, and rows of out around all of them."""
    tq, tk, pad = sum(lens_q), sum(lens_k), 70
    q, k, v = randn((tq, 4, D), 1), randn((tk, 2, D), 2), randn((tk, 2, D), 3)
    kw = dict(causal=causal)
    want = lynx.attention(q, k, v, offsets(lens_q), offsets(lens_k), **kw)

    def wide(t):
        e = spoiled(randn((pad,) + t.shape[1:], 4), slice(None))
        return torch.cat([e, t, e])

    cq, ck = offsets(lens_q) + pad, offsets(lens_k) + pad
    Q, K, V = wide(q), wide(k), wide(v)
    out, lse = nan_bf16(tuple(Q.shape)), torch.full(Q.shape[:-1], 7.0, device="cuda")
    say(f"surroundings D={D} {lens_q} causal={causal}")
    lynx.attention(Q, K, V, cq, ck, out=out, lse=lse, **kw)
    # more tokens in all: keys may be cut elsewhere, so not the bytes of the call above
    ref = ao.attention(host_f64(q), host_f64(k), host_f64(v), lens_q, lens_k, causal)
    check(out[pad:-pad], lse[pad:-pad], ref, D, max(lens_k))
    for t in (out[:pad], out[-pad:]):
        assert (t.view(torch.int16) == 0x7FC0).all()
    assert (lse[:pad] == 7).all() and (lse[-pad:] == 7).all()
    # a sequence between others that hold no number
    for s in range(3):
        a, b = sum(lens_k[:s]), sum(lens_k[:s + 1])
        others = [i for i in range(tk) if not a <= i < b]
        o = lynx.attention(q, spoiled(k, others), spoiled(v, others), offsets(lens_q), offsets(lens_k), **kw)
        i, j = sum(lens_q[:s]), sum(lens_q[:s + 1])
        assert torch.equal(o[i:j], want[i:j])


def test_query_rows_do_not_meet():
    """A row that holds no number leaves its tile's other rows as they are."""
    q, k, v = randn((200, 2, 64), 1), randn((200, 1, 64), 2), randn((200, 1, 64), 3)
    want = lynx.attention(q, k, v, causal=True)
    q[77, 1] = NAN
    q[3, 0, 5] = INF
    say("rows that hold no number")
    got = lynx.attention(q, k, v, causal=True)
    bad = torch.zeros((200, 2), dtype=torch.bool, device="cuda")
    bad[77, 1] = bad[3, 0] = True
    assert torch.isnan(got[bad]).any(-1).all()
    assert torch.equal(got[~bad], want[~bad])


@pytest.mark.parametrize("lq,lk,heads,kv", [(300, 300, 2, 2), (130, 200, 4, 1), (7, 100, 4, 1), (5, 9000, 2, 2),
                                            (600, 600, 24, 24)])
@pytest.mark.parametrize("D", [64, 72, 128])
@pytest.mark.parametrize("P", [0, 40])
def test_keys_that_are_hidden_may_hold_anything(lq, lk, heads, kv, D, P):
    """Rows before a key with NaN or infinities get the bytes they get without it; rows that see it
    what the formula gives: NaN for a key of NaN, and an infinite value in its channel alone."""
    q, k, v = randn((lq, heads, D), 1), randn((lk, kv, D), 2), randn((lk, kv, D), 3)
    prefix = (randn((P, kv, D), 4), randn((P, kv, D), 5)) if P else None
    kw = dict(causal=True, prefix=prefix, return_lse=True)
    want, wl = lynx.attention(q, k, v, **kw)
    say(f"hidden keys {lq} {lk} {heads}/{kv}x{D} P={P}")
    for i in sorted({1, lq // 2, lq - 2, lq - 1}):  # the first query that sees key j
        j = i + lk - lq
        a = v.clone()
        a[j, :, 3], a[j, :, 5], a[j, :, 6] = INF, NAN, -INF
        out, lse = lynx.attention(q, k, a, **kw)
        assert torch.equal(lse, wl)
        assert torch.equal(out[:i], want[:i])
        others = [c for c in range(D) if c not in (3, 5, 6)]
        assert torch.equal(out[..., others], want[..., others])
        assert torch.isnan(out[i:, :, 5]).all()
        # (inf p: inf, or NaN where p is 0 in bf16)
        assert not torch.isfinite(out[i:, :, 3]).any() and not (out[i:, :, 3] < 0).any()
        assert not torch.isfinite(out[i:, :, 6]).any() and not (out[i:, :, 6] > 0).any()
        b = k.clone()
        b[j] = NAN
        out, lse = lynx.attention(q, b, v, **kw)
        assert torch.equal(out[:i], want[:i]) and torch.equal(lse[:i], wl[:i])
        assert torch.isnan(out[i:]).all() and torch.isnan(lse[i:]).all()


@pytest.mark.parametrize("lq,lk,heads,kv", [(130, 200, 32, 1), (77, 333, 40, 1), (45, 130, 71, 1), (300, 300, 64, 2),
                                            (2000, 2000, 64, 2)])
@pytest.mark.parametrize("D,P", [(64, 0), (128, 40)])
def test_hidden_keys_of_rows_of_one_token(lq, lk, heads, kv, D, P):
    """With 32 heads to a key head and more all rows of a wave may be of one token, which see the same
    keys, and still not all keys of a tile.  (The last: 256-row tiles.)"""
    test_keys_that_are_hidden_may_hold_anything(lq, lk, heads, kv, D, P)


@pytest.mark.parametrize("heads", [32, 40, 71])
@pytest.mark.parametrize("D", [64, 72, 128])
def test_hidden_keys_of_few_rows_of_one_token(heads, D):
    """The same in the few-row kernel: its row tiles by the mean of sequences that have no queries too."""
    lens_q, lens_k = [2] + [0] * 12 + [3], [150, 0, 9, 1] + [0] * 9 + [33]
    q, k, v = randn((5, heads, D), 1), randn((193, 1, D), 2), randn((193, 1, D), 3)
    kw = dict(cu_q=offsets(lens_q), cu_k=offsets(lens_k), causal=True)
    want = lynx.attention(q, k, v, **kw)
    say(f"hidden keys of few rows {heads}/1x{D}")
    for key, first in ((149, 1), (191, 3), (192, 4)):  # the first row that sees the key
        seen = 2 if first < 2 else 5                   # and the first after it that does not
        a = v.clone()
        a[key, :, 3], a[key, :, 5] = INF, NAN
        out = lynx.attention(q, k, a, **kw)
        others = [i for i in range(5) if not first <= i < seen]
        assert torch.equal(out[others], want[others])
        assert torch.isnan(out[first:seen, :, 5]).all() and not torch.isfinite(out[first:seen, :, 3]).any()
        rest = [c for c in range(D) if c not in (3, 5)]
        assert torch.equal(out[..., rest], want[..., rest])


@pytest.mark.parametrize("batch,tq,tk,heads,kv", [(3, 700, 900, 4, 2), (40, 40, 5000, 8, 2), (100, 9000, 4000, 2, 2),
                                                  (9, 9, 20000, 2, 1)])
@pytest.mark.parametrize("causal,P", [(False, 0), (True, 300)])
def test_offsets_out_of_order_touch_nothing_else(batch, tq, tk, heads, kv, causal, P):
    """Offsets that decrease or lie outside are held to the tensors: what is beside out and lse stays."""
    q, k, v = randn((tq, heads, 64), 1), randn((tk, kv, 64), 2), randn((tk, kv, 64), 3)
    kw = dict(causal=causal, prefix=(randn((P, kv, 64), 4), randn((P, kv, 64), 5)) if P else None)
    rng = np.random.default_rng(batch)
    for top in (tq + 5, 2 ** 31 - 1):
        cq, ck = (torch.from_numpy(rng.integers(-top, top, batch + 1).astype(np.int32)).cuda() for _ in "qk")
        out, lse = nan_bf16((tq + 512, heads, 64)), torch.full((tq + 512, heads), 7.0, device="cuda")
        say(f"offsets in no order {batch} {tq} {tk} {top}")
        lynx.attention(q, k, v, cq, ck, out=out[256:-256], lse=lse[256:-256], **kw)
        torch.cuda.synchronize()
        for t in (out[:256], out[-256:]):
            assert (t.view(torch.int16) == 0x7FC0).all()
        assert (lse[:256] == 7).all() and (lse[-256:] == 7).all()


def test_offsets_that_go_back_and_forth():
    """32768 sequences of all tokens each: 2^31 row tiles in all, of which the launch takes a part."""
    batch, tq = 1 << 16, 1 << 21
    q, k = randn((tq, 1, 8), 1), randn((8, 1, 8), 2)
    cu = torch.zeros(batch + 1, dtype=torch.int32, device="cuda")
    cu[1::2] = tq
    out = nan_bf16((tq + 512, 1, 8))
    say("offsets back and forth")
    lynx.attention(q, k, k, cu, torch.zeros_like(cu), out=out[256:-256])
    torch.cuda.synchronize()
    for t in (out[:256], out[-256:]):
        assert (t.view(torch.int16) == 0x7FC0).all()
    assert (out[256:-256] == 0).all()  # no keys; the first sequence has all rows


# ---- offsets past 32 bits ----------------------------------------------------------

def test_a_cache_of_more_than_4_gib():
    tk, kv, D = (1 << 21) + 300, 8, 128      # 2^31 elements and more each
    say("long cache")
    k = torch.zeros((tk, kv, D), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros((tk, kv, D), dtype=torch.bfloat16, device="cuda")
    k[-300:], v[-300:] = randn((300, kv, D), 1), randn((300, kv, D), 2)
    for lq in (1, 150):
        q = randn((lq, 8, D), 3)
        ref = ao.attention(host_f64(q), host_f64(k[-300:]), host_f64(v[-300:]), [lq], [300], True)
        cq = torch.tensor([0, 0, lq], dtype=torch.int32, device="cuda")
        ck = torch.tensor([0, tk - 300, tk], dtype=torch.int32, device="cuda")
        out, lse = lynx.attention(q, k, v, cq, ck, causal=True, return_lse=True)
        check(out, lse, ref, D, 300)
    # one sequence over the whole cache: the far keys are the only ones with weight
    q = randn((1, 8, D), 3)
    k[:-300, :, 0] = -3e4
    q[..., 0] = 1.0
    ref = ao.attention(host_f64(q), host_f64(k[-300:]), host_f64(v[-300:]), [1], [300], True)
    out, lse = lynx.attention(q, k, v, causal=True, return_lse=True)
    check(out, lse, ref, D, 300)


@pytest.mark.parametrize("lq,D", [(140, 56), (140, 104), (3, 56)])
def test_the_largest_token_stride(lq, D):
    """Keys nearly 16 MiB apart: a tile of them spans nearly 2^31 bytes, and the channels behind
    head_dim, which count as zero, hold NaN here."""
    stride, lk = (1 << 23) - 8, 130
    memory = torch.full((lk * stride,), NAN, dtype=torch.bfloat16, device="cuda")
    k, v = (memory[at:].as_strided((lk, 1, D), (stride, D, 1)) for at in (0, 512))
    k.copy_(randn((lk, 1, D), 1))
    v.copy_(randn((lk, 1, D), 2))
    q = randn((lq, 1, D), 3)
    out, lse = lynx.attention(q, k, v, return_lse=True)
    check(out, lse, ao.attention(host_f64(q), host_f64(k), host_f64(v), [lq], [lk]), D, lk)


# ---- calls ------------------------------------------------------------------------

CALLS = {
    "tile": ([300, 40], [300, 40], 4, 2, 128, 0),
    "few": ([1] * 9, list(range(100, 1000, 100)), 8, 2, 128, 0),
    "prefix": ([1] * 9, list(range(1, 10)), 8, 2, 64, 500),
}


def call_inputs(name, seed):
    lq, lk, heads, kv, D, P = CALLS[name]
    t = dict(q=randn((sum(lq), heads, D), seed), k=randn((sum(lk), kv, D), seed + 1),
             v=randn((sum(lk), kv, D), seed + 2), cu_q=offsets(lq), cu_k=offsets(lk), causal=True)
    if P:
        t["prefix"] = randn((P, kv, D), seed + 3), randn((P, kv, D), seed + 4)
    return t


@pytest.mark.parametrize("name", CALLS)
def test_the_same_bytes_every_time(name):
    t = call_inputs(name, 1)
    ref = lynx.attention(return_lse=True, **t)
    lq, lk, heads, kv, D, P = CALLS[name]
    for _ in range(3):
        got = lynx.attention(**t, **poisoned(t["q"], len(lq), sum(lk), kv, P, True, True))
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


@pytest.mark.parametrize("name", CALLS)
def test_captured_and_replayed(name):
    """Two graphs with workspaces of their own, replayed with other work between, and with new
    inputs in the same tensors."""
    a, b = call_inputs(name, 1), call_inputs(name, 11)
    refs = [lynx.attention(**t).clone() for t in (a, b)]
    outs = [torch.empty_like(r) for r in refs]
    graphs = []
    say(f"capture {name}")
    for t, o in zip((a, b), outs):
        lynx.attention(out=o, **t)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            lynx.attention(out=o, **t)
        graphs.append(g)
    for _ in range(3):
        for o in outs:
            o.view(torch.int16).fill_(0x7FC0)
        for g in graphs:
            g.replay()
        junk = torch.randn((512, 512), device="cuda") @ torch.randn((512, 512), device="cuda")
        torch.cuda.synchronize()
        assert junk.isfinite().all()
        for o, r in zip(outs, refs):
            assert torch.equal(o, r)
    for n in "qkv":
        a[n].copy_(b[n])
    if "prefix" in a:
        for x, y in zip(a["prefix"], b["prefix"]):
            x.copy_(y)
    graphs[0].replay()
    assert torch.equal(outs[0], refs[1])


def test_two_streams():
    calls = [call_inputs(n, 5) for n in CALLS]
    refs = [lynx.attention(**t) for t in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    say("streams")
    outs = []
    for _ in range(4):
        outs = []
        for s, t in zip(streams, calls):
            with torch.cuda.stream(s):
                outs.append(lynx.attention(**t))
    torch.cuda.synchronize()
    for o, r in zip(outs, refs):
        assert torch.equal(o, r)
