"""lynx_attention, every row of it: the kernels for many rows (256-row tiles; few keys held in LDS) against
64 bits, head by head on the GPU, with the bounds of test_gpu_attention.py."""
import numpy as np
import pytest
import torch

import activation_sparse_gemm_amd as lynx
from tests.gpu_util import host_f64, nan_bf16, say
from tests.test_gpu_attention import check, poisoned, randn

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def reference(q, k, v, causal, prefix=None, scale=None):
    """As ao.attention, for a batch of sequences of one length [B, L, heads, D], in float64 on the GPU."""
    B, Lq, H, D = q.shape
    Lk, kv = k.shape[1:3]
    P = prefix[0].shape[0] if prefix else 0
    scale = D ** -0.5 if scale is None else scale
    out = torch.zeros((B, Lq, H, D), dtype=torch.float64, device="cuda")
    dev = torch.zeros_like(out)
    lse = torch.full((B, Lq, H), -INF, dtype=torch.float64, device="cuda")
    spread, size = torch.zeros_like(lse), torch.zeros_like(lse)
    see = torch.ones((Lq, P + Lk), dtype=torch.bool, device="cuda")
    if causal:
        see[:, P:] = torch.arange(Lk, device="cuda")[None] <= torch.arange(Lq, device="cuda")[:, None] + Lk - Lq
    some = see.any(1)
    for b in range(B):
        for h in range(H):
            Q, K, V = q[b, :, h].double(), k[b, :, h * kv // H].double(), v[b, :, h * kv // H].double()
            if P:
                K = torch.cat([prefix[0][:, h * kv // H].double(), K])
                V = torch.cat([prefix[1][:, h * kv // H].double(), V])
            Kt = K.t().contiguous()
            s = (scale * (Q @ Kt)).masked_fill(~see, -INF)
            lse[b, :, h] = torch.logsumexp(s, 1)
            p = torch.exp(s - torch.where(some, lse[b, :, h], torch.zeros_like(lse[b, :, h]))[:, None])
            o = p @ V
            out[b, :, h] = o
            dev[b, :, h] = (p @ (V * V) - o * o).clamp(min=0).sqrt()
            p2 = p * p
            size[b, :, h] = (p2 @ (V * V) - 2 * o * (p2 @ V) + o * o * p2.sum(1, keepdim=True)).sum(1).clamp(min=0).sqrt()
            spread[b, :, h] = (scale * (Q.abs() @ Kt.abs())).masked_fill(~see, 0).amax(1)
    return tuple(t.cpu().numpy() for t in (out, lse, dev, size, spread))


def run(B, lq, lk, heads, kv, D, causal, P, seed, layout="BSHD"):
    def make(L, h, s, size=1.6):
        if layout == "BHSD":
            return randn((B, h, L, D), s, size).transpose(1, 2)
        return randn((B, L, h, D), s, size)

    q, k, v = make(lq, heads, seed), make(lk, kv, seed + 1), make(lk, kv, seed + 2, 1.0)
    prefix = (randn((P, kv, D), seed + 3, 1.6), randn((P, kv, D), seed + 4)) if P else None
    say(f"every row {layout} {B}x{lq}x{lk} {heads}/{kv}x{D} causal={causal} P={P}")
    kw = poisoned(q, B, B * lk, kv, P, False, causal)
    if layout == "BHSD":
        kw["out"] = nan_bf16((B, heads, lq, D)).transpose(1, 2)
    out, lse = lynx.attention(q, k, v, causal=causal, prefix=prefix, **kw)
    ref = reference(q, k, v, causal, prefix)
    check(out, lse, ref, D, lk + P)
    # without lse another kernel: the same bytes
    again = lynx.attention(q, k, v, causal=causal, prefix=prefix)
    assert torch.equal(again, out)


# What takes 256 rows to a tile: many rows, whether the keys are cut (4096 x 16 heads, causal; 299 x 40 heads) or not
MANY = [(1, 4096, 4096, 16, 16, 0), (1, 4095, 4093, 16, 16, 100), (1, 2001, 2000, 64, 2, 0), (1, 299, 20001, 40, 4, 0),
        (3, 1501, 30000, 32, 4, 0), (1, 5000, 3000, 32, 16, 70)]


@pytest.mark.parametrize("B,lq,lk,heads,kv,P", MANY)
@pytest.mark.parametrize("D", [64, 72, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_256_row_tiles(B, lq, lk, heads, kv, P, D, causal):
    run(B, lq, lk, heads, kv, D, causal, P, 1)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("layout", ["BSHD", "BHSD"])
def test_256_row_tiles_on_a_prefix_of_a_batch(causal, layout):
    run(4, 1024, 1024, 24, 24, 128, causal, 2560, 2, layout)
    run(1, 4090, 4096, 16, 16, 80, causal, 65, 3, layout)


@pytest.mark.parametrize("B,lq,lk,heads,kv,D", [
    (2, 4100, 300, 16, 16, 72), (3, 3001, 640, 12, 12, 64), (1, 9000, 320, 14, 2, 128), (70, 131, 33, 16, 8, 96),
    (5, 2011, 1, 16, 4, 128), (1, 8200, 65, 32, 8, 128),
])
@pytest.mark.parametrize("layout", ["BSHD", "BHSD"])
def test_many_rows_on_few_keys(B, lq, lk, heads, kv, D, layout):
    run(B, lq, lk, heads, kv, D, False, 0, 4, layout)


CALLS = {"wide": (1, 2000, 2000, 64, 2, 128, False), "wide causal": (1, 4096, 4096, 16, 16, 64, True),
         "few keys": (2, 4100, 300, 16, 16, 72, False)}


@pytest.mark.parametrize("name", CALLS)
def test_the_same_bytes_from_a_graph(name):
    B, lq, lk, heads, kv, D, causal = CALLS[name]
    q, k, v = randn((B, lq, heads, D), 1), randn((B, lk, kv, D), 2), randn((B, lk, kv, D), 3)
    say(f"graph {name}")
    want = lynx.attention(q, k, v, causal=causal)
    out = torch.empty_like(want)
    lynx.attention(q, k, v, causal=causal, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lynx.attention(q, k, v, causal=causal, out=out)
    for _ in range(3):
        out.view(torch.int16).fill_(0x7FC0)
        g.replay()
        junk = torch.randn((512, 512), device="cuda") @ torch.randn((512, 512), device="cuda")
        torch.cuda.synchronize()
        assert junk.isfinite().all() and torch.equal(out, want)
        assert torch.equal(lynx.attention(q, k, v, causal=causal), want)
    q.copy_(randn((B, lq, heads, D), 4))
    g.replay()
    assert torch.equal(out, lynx.attention(q, k, v, causal=causal))


@pytest.mark.parametrize("D,lk", [(72, 300), (64, 500), (128, 65)])
def test_values_that_are_no_numbers_on_few_keys(D, lk):
    """A key or value of one sequence reaches all rows of that sequence and head, in the value's
    channel alone; a query row reaches itself."""
    B, lq, heads = 3, 2500, 16
    q, k, v = randn((B, lq, heads, D), 1), randn((B, lk, heads, D), 2), randn((B, lk, heads, D), 3)
    want = lynx.attention(q, k, v)
    say(f"few keys that are no numbers {lk}x{D}")
    a = v.clone()
    a[1, lk - 1, 2, 3], a[1, 0, 3, 5] = INF, NAN
    out = lynx.attention(q, k, a)
    hit = torch.zeros((B, lq, heads, D), dtype=torch.bool, device="cuda")
    hit[1, :, 2, 3] = hit[1, :, 3, 5] = True
    assert not torch.isfinite(out[hit]).any() and torch.isnan(out[1, :, 3, 5]).all()
    assert torch.equal(out[~hit], want[~hit])
    b, c = k.clone(), q.clone()
    b[2, lk // 2, 7] = NAN
    c[0, 2499, 15], c[0, 31, 0, 1] = NAN, INF
    out = lynx.attention(c, b, v)
    hit = torch.zeros((B, lq, heads), dtype=torch.bool, device="cuda")
    hit[2, :, 7] = hit[0, 2499, 15] = hit[0, 31, 0] = True
    assert torch.isnan(out[hit]).all(-1).sum() >= hit.sum() - 1 and torch.isnan(out[0, 31, 0]).any()
    assert torch.equal(out[~hit], want[~hit])


@pytest.mark.parametrize("D", [64, 72, 128])
def test_hidden_keys_of_256_row_tiles(D):
    lq, lk, heads, P = 4096, 4099, 16, 40
    q, k, v = randn((lq, heads, D), 1), randn((lk, heads, D), 2), randn((lk, heads, D), 3)
    prefix = randn((P, heads, D), 4), randn((P, heads, D), 5)
    kw = dict(causal=True, prefix=prefix, return_lse=True)
    want, wl = lynx.attention(q, k, v, **kw)
    say(f"hidden keys of 256-row tiles {D}")
    others = [c for c in range(D) if c not in (3, 5)]
    for i in (1, 255, 2048, 3001, lq - 1):
        a, b = v.clone(), k.clone()
        a[i + lk - lq, :, 3], a[i + lk - lq, :, 5] = -INF, NAN
        b[i + lk - lq] = NAN
        out, lse = lynx.attention(q, k, a, **kw)
        assert torch.equal(lse, wl) and torch.equal(out[:i], want[:i])
        assert torch.equal(out[..., others], want[..., others])
        assert torch.isnan(out[i:, :, 5]).all() and not torch.isfinite(out[i:, :, 3]).any()
        out, lse = lynx.attention(q, b, v, **kw)
        assert torch.equal(out[:i], want[:i]) and torch.equal(lse[:i], wl[:i])
        assert torch.isnan(out[i:]).all() and torch.isnan(lse[i:]).all()
