"""The 8-bit linear layer, its quantisers and the block norms: what is timed and what the results are.

`listed()` and `draw(rng)` give cases, `prepare(case, seed)` a case's inputs on the GPU, and `run(state)` one pass,
through the library's entry points where `own` is true and else in elementary torch operations in 32 bits.
`work(case)` is the least a pass has to move and compute, `exact(case, seed)` its result in 64 bits.

The 8-bit operand: values e4m3, one power-of-two scale (an E8M0 byte, 2^(byte - 127)) for each 128 consecutive
channels of an activation's row, and for each block of 128 rows x 128 channels of a weight.  Activation scales are
stored as [ceil(K / 512), M, 4] (four blocks of a row to a 32-bit word), weight scales as
[ceil(N / 128), ceil(K / 128) rounded up to 4]; unused places hold 127.
"""
import math

import torch

own = False

BLOCK = 128
TOP = 448.0  # the largest e4m3 value


# ---- cases -------------------------------------------------------------------------------------------------------

def listed():
    return [
        # quantising an activation: a short ragged batch with a half-filled last block ...
        {"name": "quantize 333x1472", "op": "quantize", "M": 333, "K": 1472},
        # ... and the MLP's wide hidden activation of a guidance-batched block
        {"name": "quantize 9216x12288", "op": "quantize", "M": 9216, "K": 12288},
        # a checkpoint's QKV weight, quantised when it is loaded
        {"name": "quantize weight 9216x3072", "op": "quantize_weight", "N": 9216, "K": 3072},
        # the whole layer: the modulation projection of one conditioning vector per sample (two samples)
        {"name": "linear 2x3072->18432", "op": "linear", "M": 2, "K": 3072, "N": 18432},
        # text tokens of one prompt through a QKV projection
        {"name": "linear 77x3072->9216", "op": "linear", "M": 77, "K": 3072, "N": 9216},
        # sizes that divide nothing
        {"name": "linear 1000x1472->1102", "op": "linear", "M": 1000, "K": 1472, "N": 1102},
        # the output projection to patches: many rows, few columns
        {"name": "linear 4096x3072->64", "op": "linear", "M": 4096, "K": 3072, "N": 64},
        # MLP-up of one image, quantised on the way in
        {"name": "linear 4096x3072->12288", "op": "linear", "M": 4096, "K": 3072, "N": 12288},
        # the product alone, on an operand that is in hand: the block's MLP-down
        {"name": "product 9216x12288->3072", "op": "product", "M": 9216, "K": 12288, "N": 3072},
        # a pre-norm with modulation on a few rows (latency)
        {"name": "norm 64x3072", "op": "norm", "M": 64, "C": 3072, "B": 2, "norm": "layer", "post": "no branch",
         "fp32": False, "fp8": False, "affine": False},
        # after a branch: post-norm, gate, fp32 residual stream, then the next norm, to bf16
        {"name": "residual norm 4096x3072", "op": "norm", "M": 4096, "C": 3072, "B": 1, "norm": "rms", "post": "rms",
         "fp32": True, "fp8": False, "affine": True},
        # the path between two layers: gate + residual + next norm into the 8-bit operand, then MLP-up on it
        {"name": "norm+linear 9216x3072->12288", "op": "norm_linear", "M": 9216, "C": 3072, "N": 12288, "B": 2,
         "norm": "layer", "post": "none", "fp32": False, "fp8": True, "affine": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "quantize_weight", "linear", "linear", "linear", "product", "norm", "norm",
                     "norm_linear"])
    K = 64 * _log(rng, 1, 192)
    if op == "quantize":
        return {"op": op, "M": _log(rng, 1, 9216), "K": K}
    if op == "quantize_weight":
        return {"op": op, "N": _log(rng, 16, 12288), "K": K}
    if op in ("linear", "product"):
        M = _log(rng, 1, 9216)
        return {"op": op, "M": M, "K": K, "N": min(_log(rng, 16, 18432), 9216 * 12288 * 3072 // (M * K))}
    B = rng.choice([1, 2, 3])
    fp8 = op == "norm_linear" or rng.random() < 0.3
    C = 64 * _log(rng, 1, 64) if fp8 else 8 * _log(rng, 2, 512)
    case = {"op": "norm_linear" if fp8 else op, "M": B * _log(rng, 1, 4096), "C": C, "B": B,
            "norm": rng.choice(["rms", "layer"]), "post": rng.choice(["none", "rms", "layer"]) if fp8 else
            rng.choice(["none", "rms", "layer", "no branch"]), "fp32": rng.random() < 0.5, "fp8": fp8,
            "affine": rng.random() < 0.5}
    if fp8:
        case["N"] = _log(rng, 64, 9216)
    return case


def work(case):
    op = case["op"]
    if op == "quantize":
        n = case["M"] * case["K"]
        return {"bytes": 3 * n + n // BLOCK, "flops": 3 * n}
    if op == "quantize_weight":
        n = case["N"] * case["K"]
        return {"bytes": 3 * n + n // BLOCK ** 2, "flops": 3 * n}
    if op in ("linear", "product"):
        M, K, N = case["M"], case["K"], case["N"]
        x = 2 * M * K if op == "linear" else M * K + M * K // BLOCK
        return {"bytes": x + N * K + N * K // BLOCK ** 2 + 2 * M * N, "flops": 2 * M * N * K}
    M, C = case["M"], case["C"]
    x = (4 if case["fp32"] else 2) * M * C
    branch = case["post"] != "no branch"
    b = x + (2 * M * C + x if branch else 0) + (M * C + M * C // BLOCK if case["fp8"] else 2 * M * C)
    b += 2 * C * (case["B"] * (3 if branch else 2) + (2 if case["affine"] else 0))
    f = 12 * M * C
    if op == "norm_linear":
        b += case["N"] * C + case["N"] * C // BLOCK ** 2 + 2 * M * case["N"]
        f += 2 * M * case["N"] * C
    return {"bytes": b, "flops": f}


# ---- inputs ------------------------------------------------------------------------------------------------------

def _activation(M, K, g):
    """Heavy-tailed, with channel scales of their own and a few channels far above the rest."""
    u = torch.rand((M, K), device="cuda", generator=g) - 0.5
    c = torch.randn((K,), device="cuda", generator=g).exp()
    c = c * torch.where(torch.rand((K,), device="cuda", generator=g) < 0.01, 20.0, 1.0)
    return (-u.sign() * torch.log1p(-2 * u.abs().clamp(max=0.4999999)) * c).to(torch.bfloat16)


def _weight(N, K, g):
    return (torch.randn((N, K), device="cuda", generator=g) * K ** -0.5).to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, s = case["op"], {"case": dict(case)}
    if op == "quantize":
        s["X"] = _activation(case["M"], case["K"], g)
    elif op == "quantize_weight":
        s["W"] = _weight(case["N"], case["K"], g)
    elif op in ("linear", "product"):
        s["X"] = _activation(case["M"], case["K"], g)
        s["Wq"], s["Ws"] = _quantize_weight(_weight(case["N"], case["K"], g))
        if op == "product":
            s["Xq"], s["Xs"] = _quantize(s.pop("X").float())
    else:
        M, C, B = case["M"], case["C"], case["B"]
        s["x"] = _activation(M, C, g)
        if case["fp32"]:
            s["x"] = s["x"].float() * (1 + 1e-3 * torch.rand((M, C), device="cuda", generator=g))
        if case["post"] != "no branch":
            s["y"] = _activation(M, C, g)
        # shift, scale and gate of one sample side by side, as a modulation projection writes them
        mod = (0.3 * torch.randn((B, 3, C), device="cuda", generator=g)).to(torch.bfloat16)
        s["shift"], s["scale"], s["gate"] = mod[:, 0], mod[:, 1], mod[:, 2]
        if case["affine"]:
            for k in ("weight", "post_weight"):
                s[k] = (1 + 0.2 * torch.randn((C,), device="cuda", generator=g)).to(torch.bfloat16)
        if op == "norm_linear":
            s["Wq"], s["Ws"] = _quantize_weight(_weight(case["N"], C, g))
    return s


# ---- one pass ----------------------------------------------------------------------------------------------------

def run(s):
    c = s["case"]
    return _run_own(c, s) if own else _run_plain(c, s)


def _run_own(c, s):
    import activation_sparse_gemm_amd as lynx
    op = c["op"]
    if op == "quantize":
        q, e = lynx.quantize_fp8(s["X"])
        return q, e.view(torch.uint8)
    if op == "quantize_weight":
        q, e = lynx.quantize_fp8_weight(s["W"])
        return q, e.view(torch.uint8)
    if op == "linear":
        return lynx.linear_fp8(s["X"], s["Wq"], s["Ws"])
    if op == "product":
        return lynx.linear_fp8_packed(s["Xq"], s["Xs"], s["Wq"], s["Ws"])
    mod = dict(norm=c["norm"], weight=s.get("weight"), scale=s["scale"], shift=s["shift"], fp8=c["fp8"])
    if c["post"] == "no branch":
        return lynx.norm_modulate(s["x"], **mod)
    x, h = lynx.residual_norm(s["x"], s["y"], gate=s["gate"], post_norm=None if c["post"] == "none" else c["post"],
                              post_weight=s.get("post_weight") if c["post"] != "none" else None, **mod)
    return (x, lynx.linear_fp8_packed(*h, s["Wq"], s["Ws"])) if op == "norm_linear" else (x, h)


def _exponents(top):
    """The smallest e with top <= 448 2^e (448 = 7/8 2^9), from the fraction and exponent of `top`."""
    frac, ex = torch.frexp(top)
    e = torch.where(frac <= 0.875, ex - 9, ex - 8).clamp(-127, 127)
    return torch.where(top == 0, torch.zeros_like(e), e)


def _quantize(x):
    """x [M, K] in 32 bits -> e4m3 values [M, K], scale bytes [ceil(K / 512), M, 4] as E8M0."""
    M, K = x.shape
    kb = -(-K // BLOCK)
    t = torch.nn.functional.pad(x, (0, kb * BLOCK - K)).view(M, kb, BLOCK)
    e = _exponents(t.abs().amax(-1))
    q = torch.ldexp(t, -e[..., None]).view(M, kb * BLOCK)[:, :K].contiguous().to(torch.float8_e4m3fn)
    b = torch.nn.functional.pad((e + 127).to(torch.uint8), (0, -kb % 4), value=127)
    return q, b.view(M, -1, 4).transpose(0, 1).contiguous().view(torch.float8_e8m0fnu)


def _quantize_weight(W):
    N, K = W.shape
    nb, kb = -(-N // BLOCK), -(-K // BLOCK)
    t = torch.nn.functional.pad(W.float(), (0, kb * BLOCK - K, 0, nb * BLOCK - N)).view(nb, BLOCK, kb, BLOCK)
    e = _exponents(t.abs().amax(dim=(1, 3)))
    q = torch.ldexp(t, -e[:, None, :, None]).view(nb * BLOCK, kb * BLOCK)[:N, :K].contiguous().to(torch.float8_e4m3fn)
    b = torch.nn.functional.pad((e + 127).to(torch.uint8), (0, -kb % 4), value=127)
    return q, b.view(torch.float8_e8m0fnu)


def _values(q, exps):
    """What an operand stands for, in 32 bits: exps [rows, blocks] of integers."""
    return torch.ldexp(q.float(), exps.repeat_interleave(BLOCK, 1)[:, :q.shape[1]])


def _product(Xq, Xs, Wq, Ws):
    x = _values(Xq, (Xs.view(torch.uint8).int() - 127).transpose(0, 1).reshape(Xq.shape[0], -1))
    w = _values(Wq, (Ws.view(torch.uint8).int() - 127).repeat_interleave(BLOCK, 0)[:Wq.shape[0]])
    return torch.matmul(x, w.t()).to(torch.bfloat16)


def _norm(t, kind, weight):
    if kind == "none":
        return t
    if kind == "layer":
        t = t - t.mean(-1, keepdim=True)
    t = t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6)
    return t if weight is None else t * weight.float()


def _run_plain(c, s):
    op = c["op"]
    if op == "quantize":
        q, e = _quantize(s["X"].float())
        return q, e.view(torch.uint8)
    if op == "quantize_weight":
        q, e = _quantize_weight(s["W"])
        return q, e.view(torch.uint8)
    if op == "linear":
        return _product(*_quantize(s["X"].float()), s["Wq"], s["Ws"])
    if op == "product":
        return _product(s["Xq"], s["Xs"], s["Wq"], s["Ws"])
    M, C, B = c["M"], c["C"], c["B"]
    x = s["x"].float().view(B, M // B, C)
    branch = c["post"] != "no branch"
    if branch:
        z = _norm(s["y"].float().view(B, M // B, C), c["post"], s.get("post_weight"))
        x = x + s["gate"].float()[:, None] * z
    h = _norm(x, c["norm"], s.get("weight")) * (1 + s["scale"].float()[:, None]) + s["shift"].float()[:, None]
    h, x = h.view(M, C), x.view(M, C).to(s["x"].dtype)
    h = _product(*_quantize(h), s["Wq"], s["Ws"]) if op == "norm_linear" else h.to(torch.bfloat16)
    return (x, h) if branch else h


# ---- the same in 64 bits, from the definitions -------------------------------------------------------------------

def _scales64(top):
    """2^e with the smallest e that keeps top / 2^e at 448 or below."""
    e = torch.ceil(torch.log2(top / TOP))
    e = torch.where(torch.exp2(e - 1) * TOP >= top, e - 1, e)
    e = torch.where(torch.exp2(e) * TOP < top, e + 1, e)
    return torch.where(top > 0, torch.exp2(e.clamp(-127, 127)), torch.ones_like(top))


def _e4m3(v):
    """v (|v| <= 448) to the nearest e4m3 value, ties to even: 3 fraction bits, exponents from -6."""
    _, ex = torch.frexp(v)
    step = torch.exp2((ex - 1).clamp(min=-6).double() - 3)
    return torch.round(v / step) * step


def _blocks64(x):
    kb = -(-x.shape[1] // BLOCK)
    return [x[:, BLOCK * i:BLOCK * (i + 1)] for i in range(kb)]


def _quantize64(x):
    """(values before scaling, values) of an activation."""
    scale = torch.stack([_scales64(t.abs().amax(1)) for t in _blocks64(x)], 1)
    wide = scale.repeat_interleave(BLOCK, 1)[:, :x.shape[1]]
    q = _e4m3(x / wide)
    return q, q * wide, scale


def _weight64(s):
    """The weight that an operand in hand stands for."""
    e = s["Ws"].view(torch.uint8).double() - 127
    i = torch.arange(s["Wq"].shape[0], device="cuda") // BLOCK
    k = torch.arange(s["Wq"].shape[1], device="cuda") // BLOCK
    return s["Wq"].double() * torch.exp2(e[i][:, k])


def _norm64(t, kind, weight):
    if kind == "none":
        return t
    if kind == "layer":
        t = t - t.sum(1, keepdim=True) / t.shape[1]
    t = t / torch.sqrt((t * t).sum(1, keepdim=True) / t.shape[1] + 1e-6)
    return t if weight is None else t * weight.double()


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "quantize":
        q, _, scale = _quantize64(s["X"].double())
        return q, None
    if op == "quantize_weight":
        W = s["W"].double()
        top = torch.stack([torch.stack([b.abs().max() for b in t.split(BLOCK, 0)]) for t in _blocks64(W)], 1)
        i = torch.arange(W.shape[0], device="cuda") // BLOCK
        k = torch.arange(W.shape[1], device="cuda") // BLOCK
        return _e4m3(W / _scales64(top)[i][:, k]), None
    if op == "linear":
        return _quantize64(s["X"].double())[1] @ _weight64(s).t()
    if op == "product":
        e = s["Xs"].view(torch.uint8).double() - 127
        k = torch.arange(case["K"], device="cuda") // BLOCK
        return (s["Xq"].double() * torch.exp2(e[k // 4, :, k % 4].t())) @ _weight64(s).t()
    x, branch = s["x"].double(), case["post"] != "no branch"
    per = torch.arange(case["M"], device="cuda") // (case["M"] // case["B"])
    if branch:
        x = x + s["gate"].double()[per] * _norm64(s["y"].double(), case["post"], s.get("post_weight"))
    h = _norm64(x, case["norm"], s.get("weight")) * (1 + s["scale"].double()[per]) + s["shift"].double()[per]
    if op == "norm_linear":
        h = _quantize64(h)[1] @ _weight64(s).t()
    return (x, h) if branch else h
