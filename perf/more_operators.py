"""The attention half of a block - rotary positions of q and k, attention, attention with a prefix that the batch
shares: what is timed and what the results are.

`listed()` and `draw(rng)` give cases, `prepare(case, seed)` a case's inputs on the GPU, and `run(state)` one pass,
through the library's entry points where `own` is true and else in elementary torch operations in 32 bits (angles in
64).  `work(case)` is the least a pass has to move and compute, `exact(case, seed)` its result in 64 bits.

rotary.  x [D] of one token and head, normed before by its rms where `norm` is true.  Axis a has d_a channels; pair i
of the R / 2 pairs (R = sum of d_a) is place j of axis a and turns by

    positions[t, a] * theta ** (-2 j / d_a)      ladder "axis":  each axis has its own frequencies
    positions[t, a] * theta ** (-2 i / R)        ladder "joint": the axes share one row of frequencies

A pair is channels (2 i, 2 i + 1) ("adjacent") or (i, i + R / 2) ("halves"); channels from R on are not turned.

attention.  Query i of a sequence of Lq queries and Lk keys sees every key of the prefix and own keys j, all of them or
(causal) those with j <= i + Lk - Lq.  Head h reads key head h // (heads / kv_heads).  out = softmax(scale q k^T) v,
lse = log of the sum of exponentials; a query that sees no key has out = 0 and lse = -inf.
"""
import math

import torch

own = False


# ---- cases -------------------------------------------------------------------------------------------------------
# Lengths of sequences are texts: "5,0,77".  "same" keys: as many as queries.  A batch of equal lengths is given as
# 4-D tensors ("batched"), one of different lengths packed into 3-D tensors with offsets.

def listed():
    return [
        # the newest token of a stream, one axis, far from the start: latency
        {"name": "rotary 1x32+8", "op": "rotary", "T": 1, "heads": 32, "kv_heads": 8, "D": 128, "axes": "128",
         "theta": 1e6, "pairs": "halves", "ladder": "axis", "norm": False, "float": False, "far": 1000000},
        # text and image tokens of one picture, with the norm of q and k before
        {"name": "rotary 4608x24+24", "op": "rotary", "T": 4608, "heads": 24, "kv_heads": 24, "D": 128,
         "axes": "16,56,56", "theta": 1e4, "pairs": "adjacent", "ladder": "axis", "norm": True, "float": False,
         "far": 64},
        # an odd number of video tokens, narrow heads, some channels not turned, positions that are scaled
        {"name": "rotary 8191x16+16 of 72", "op": "rotary", "T": 8191, "heads": 16, "kv_heads": 16, "D": 72,
         "axes": "16,24,24", "theta": 1e4, "pairs": "halves", "ladder": "axis", "norm": True, "float": True,
         "far": 256},
        # a long packed prompt of text, images and video, one row of frequencies for its three axes, grouped heads
        {"name": "rotary 20000x28+4", "op": "rotary", "T": 20000, "heads": 28, "kv_heads": 4, "D": 128,
         "axes": "32,48,48", "theta": 1e6, "pairs": "halves", "ladder": "joint", "norm": False, "float": False,
         "far": 30000},
        # a short prompt through a text encoder: latency
        {"name": "attention 77 causal 12x64", "op": "attention", "q": "77", "k": "same", "prefix": 0, "heads": 12,
         "kv_heads": 12, "D": 64, "causal": True, "batched": False, "lse": False},
        # text and image tokens of one picture
        {"name": "attention 4608 24x128", "op": "attention", "q": "4608", "k": "same", "prefix": 0, "heads": 24,
         "kv_heads": 24, "D": 128, "causal": False, "batched": True, "lse": False},
        # image tokens on the prompt's tokens, a guided pair, a head size that is no power of two
        {"name": "attention 2x4096 on 300 16x72", "op": "attention", "q": "4096,4096", "k": "300,300", "prefix": 0,
         "heads": 16, "kv_heads": 16, "D": 72, "causal": False, "batched": True, "lse": False},
        # prompts of different lengths in one batch, one of them empty, grouped heads
        {"name": "attention packed causal 32/8x128", "op": "attention", "q": "1,777,4173,0,33,2048,129,1500",
         "k": "same", "prefix": 0, "heads": 32, "kv_heads": 8, "D": 128, "causal": True, "batched": False,
         "lse": True},
        # one long prompt
        {"name": "attention 16384 causal 32/8x128", "op": "attention", "q": "16384", "k": "same", "prefix": 0,
         "heads": 32, "kv_heads": 8, "D": 128, "causal": True, "batched": False, "lse": False},
        # the next token of 32 streams, caches of different lengths
        {"name": "attention 32 tokens on caches 32/8x128", "op": "attention", "q": ",".join(["1"] * 32),
         "k": ",".join(str(17 + (i * 5273) % 16384) for i in range(32)), "prefix": 0, "heads": 32, "kv_heads": 8,
         "D": 128, "causal": True, "batched": False, "lse": False},
        # the next token of 48 streams that began with the same long text
        {"name": "prefix 8192, 48 tokens 32/8x128", "op": "prefix", "q": ",".join(["1"] * 48),
         "k": ",".join(str(1 + (i * 97) % 512) for i in range(48)), "prefix": 8192, "heads": 32, "kv_heads": 8,
         "D": 128, "causal": True, "batched": False, "lse": True},
        # four pictures from one prompt and one reference picture, whose keys and values are kept
        {"name": "prefix 2560, 4x1024 24x128", "op": "prefix", "q": "1024,1024,1024,1024", "k": "same",
         "prefix": 2560, "heads": 24, "kv_heads": 24, "D": 128, "causal": False, "batched": True, "lse": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_rotary(rng):
    D = rng.choice([32, 64, 72, 80, 96, 128])
    left, axes = D, []
    for _ in range(rng.choice([1, 2, 3])):
        if left >= 2:
            axes.append(2 * rng.randint(1, left // 2))
            left -= axes[-1]
    kv = rng.choice([1, 2, 4, 8, 12, 16, 24])
    heads = kv * rng.choice([1, 1, 2, 4])
    return {"op": "rotary", "T": min(_log(rng, 1, 40000), 80000000 // ((heads + kv) * D)), "heads": heads,
            "kv_heads": kv, "D": D, "axes": ",".join(map(str, axes)), "theta": rng.choice([256.0, 1e4, 1e6]),
            "pairs": rng.choice(["adjacent", "halves"]), "ladder": rng.choice(["axis", "joint"]),
            "norm": rng.random() < 0.5, "float": rng.random() < 0.3, "far": _log(rng, 16, 1000000)}


def draw(rng):
    op = rng.choice(["rotary", "rotary", "attention", "attention", "attention", "prefix", "prefix"])
    if op == "rotary":
        return _draw_rotary(rng)
    D = rng.choice([32, 64, 72, 80, 96, 128, 128])
    kv = rng.choice([1, 2, 4, 8, 12, 16, 24])
    heads = kv * rng.choice([1, 1, 2, 4, 7, 8])
    B = _log(rng, 1, 48)
    kind = rng.choice(["self", "self", "cross", "tokens", "tokens"])
    batched = rng.random() < 0.4

    def lengths(top):
        top = max(1, top)
        if batched:
            return [_log(rng, 1, top)] * B
        return [0 if B > 1 and rng.random() < 0.04 else _log(rng, 1, top) for _ in range(B)]

    prefix = _log(rng, 1, 8192) if op == "prefix" else 0
    budget = 4 * 10 ** 9  # visible pairs times heads: the largest listed case has 4.3e9
    if kind == "tokens":
        q = [rng.choice([1, 1, 1, 2, 5, 16])] * B
        k = lengths(min(32768, 2 ** 19 // (B * kv) * 8))
        k = [max(a, b) for a, b in zip(q, k)]
    else:
        q = lengths(min(8192, int(math.sqrt(budget / (heads * B))), budget // (heads * B * (prefix + 1))))
        k = q if kind == "self" else lengths(1024)
        if kind == "self" and rng.random() < 0.3:
            k = [a + rng.randint(0, 500) for a in q] if not batched else [q[0] + rng.randint(0, 500)] * B
    if sum(q) == 0:
        return draw(rng)
    return {"op": op, "q": ",".join(map(str, q)), "k": "same" if k is q else ",".join(map(str, k)),
            "prefix": prefix, "heads": heads, "kv_heads": kv, "D": D, "causal": kind != "cross" and rng.random() < 0.7,
            "batched": batched, "lse": (op == "prefix" or min(k) > 0) and rng.random() < 0.4}


def _lengths(case):
    q = [int(n) for n in case["q"].split(",")]
    return q, q if case["k"] == "same" else [int(n) for n in case["k"].split(",")]


def _seen(lq, lk, causal):
    """Pairs of a query and an own key that it sees."""
    if not causal:
        return lq * lk
    n = min(lq, lk)  # the last n queries see lk - n + 1 .. lk keys
    return n * (lk - n) + n * (n + 1) // 2


def work(case):
    if case["op"] == "rotary":
        n = case["T"] * (case["heads"] + case["kv_heads"]) * case["D"]
        b = 4 * n + 4 * case["T"] * len(case["axes"].split(",")) + (4 * case["D"] if case["norm"] else 0)
        return {"bytes": b, "flops": n * (7 if case["norm"] else 3)}
    q, k = _lengths(case)
    D, H, P = case["D"], case["heads"], case["prefix"]
    pairs = sum(_seen(a, b, case["causal"]) + a * P for a, b in zip(q, k))
    b = 4 * sum(q) * H * D + 4 * (sum(k) + P) * case["kv_heads"] * D
    b += 4 * sum(q) * H if case["lse"] else 0
    b += 0 if case["batched"] else 8 * (len(q) + 1)
    return {"bytes": b, "flops": 4 * D * H * pairs}


# ---- inputs ------------------------------------------------------------------------------------------------------

def _bf16(shape, g, size=1.0):
    return (size * torch.randn(shape, device="cuda", generator=g)).to(torch.bfloat16)


def _positions(case, g):
    """A raster of places (the last axis fastest) that starts at a random place below `far` on the first axis."""
    axes = case["axes"].split(",")
    side = max(1, math.isqrt(case["T"]) if len(axes) < 3 else round(case["T"] ** (1 / 3)) * 2)
    t = torch.arange(case["T"], device="cuda")
    cols = []
    for _ in axes[1:]:
        cols.insert(0, t % side)
        t = t // side
    cols.insert(0, t + torch.randint(0, case["far"], (1,), device="cuda", generator=g))
    p = torch.stack(cols, 1)
    if case["float"]:
        return (p.float() * (0.5 + torch.rand((1, len(axes)), device="cuda", generator=g))).contiguous()
    return p.to(torch.int32).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = {"case": dict(case)}
    H, kv, D = case["heads"], case["kv_heads"], case["D"]
    if case["op"] == "rotary":
        # one projection's output: heads of q, of k and of v side by side
        qkv = _bf16((case["T"], H + 2 * kv, D), g)
        qkv *= torch.exp(0.5 * torch.randn((1, H + 2 * kv, 1), device="cuda", generator=g)).to(torch.bfloat16)
        s["q"], s["k"] = qkv[:, :H], qkv[:, H:H + kv]
        s["positions"], s["axes"] = _positions(case, g), tuple(int(a) for a in case["axes"].split(","))
        if case["norm"]:
            for n in ("q_weight", "k_weight"):
                s[n] = (1 + 0.2 * torch.randn((D,), device="cuda", generator=g)).to(torch.bfloat16)
        return s
    q, k = _lengths(case)
    # q and k as they come out of their norms (scores of a spread of about 2.5), v as it comes out of a projection
    s["q"], s["k"] = _bf16((sum(q), H, D), g, 1.6), _bf16((sum(k), kv, D), g, 1.6)
    s["v"] = _bf16((sum(k), kv, D), g)
    if case["batched"]:
        for n, l in (("q", q), ("k", k), ("v", k)):
            s[n] = s[n].view(len(l), l[0], -1, D)
    else:
        for n, l in (("cu_q", q), ("cu_k", k)):
            s[n] = torch.tensor([sum(l[:i]) for i in range(len(l) + 1)], dtype=torch.int32, device="cuda")
    if case["prefix"]:
        s["prefix"] = _bf16((case["prefix"], kv, D), g, 1.6), _bf16((case["prefix"], kv, D), g)
    return s


# ---- one pass ----------------------------------------------------------------------------------------------------

def run(s):
    c = s["case"]
    return _run_own(c, s) if own else _run_plain(c, s)


def _run_own(c, s):
    import activation_sparse_gemm_amd as lynx
    if c["op"] == "rotary":
        return lynx.qk_rotary(s["q"], s["k"], s["positions"], s["axes"], theta=c["theta"], pairs=c["pairs"],
                              ladder=c["ladder"], norm="rms" if c["norm"] else None, q_weight=s.get("q_weight"),
                              k_weight=s.get("k_weight"))
    return lynx.attention(s["q"], s["k"], s["v"], cu_q=s.get("cu_q"), cu_k=s.get("cu_k"), causal=c["causal"],
                          prefix=s.get("prefix"), return_lse=c["lse"])


def _run_plain(c, s):
    if c["op"] == "rotary":
        return _rotary_plain(c, s)
    q, k = _lengths(c)
    H, D = c["heads"], c["D"]
    Q, K, V = (s[n].reshape(-1, s[n].shape[-2], D).transpose(0, 1).float() for n in "qkv")
    out = torch.empty((sum(q), H, D), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((sum(q), H), device="cuda")
    prefix = [t.transpose(0, 1).float() for t in s["prefix"]] if c["prefix"] else None
    i = j = 0
    for lq, lk in zip(q, k):
        if lq:
            k_s, v_s = K[:, j:j + lk], V[:, j:j + lk]
            if prefix:
                k_s, v_s = torch.cat([prefix[0], k_s], 1), torch.cat([prefix[1], v_s], 1)
            out[i:i + lq], lse[i:i + lq] = _attention_plain(Q[:, i:i + lq], k_s, v_s, lk, c["causal"])
        i, j = i + lq, j + lk
    shape = s["q"].shape
    return (out.view(shape), lse.view(shape[:-1])) if c["lse"] else out.view(shape)


def _attention_plain(q, k, v, lk, causal):
    """q [H, lq, D], k and v [kv_heads, prefix + lk, D] in 32 bits -> out [lq, H, D], lse [lq, H]."""
    (H, lq, D), (kv, n, _) = q.shape, k.shape
    G = H // kv
    q = q.reshape(kv, G * lq, D)
    hidden = None
    if causal and lq > 1:
        last = torch.arange(lq, device="cuda") + (lk - lq) + (n - lk)
        hidden = torch.arange(n, device="cuda")[None] > last[:, None]
        hidden[:, :n - lk] = False
    o, z = torch.empty_like(q), torch.empty((kv, G * lq), device="cuda")
    step = max(1, (1 << 30) // max(1, G * lq * n))  # key heads at once: scores of 4 GiB at most
    for h in range(0, kv, step):
        x = torch.matmul(q[h:h + step], k[h:h + step].transpose(1, 2).contiguous()) * D ** -0.5
        if hidden is not None:
            x.view(-1, G, lq, n).masked_fill_(hidden, -math.inf)
        if n == 0:
            o[h:h + step], z[h:h + step] = 0, -math.inf
            continue
        m = x.amax(-1, keepdim=True)
        m = torch.where(m == -math.inf, torch.zeros_like(m), m)
        x = x.sub_(m).exp_()
        t = x.sum(-1, keepdim=True)
        z[h:h + step] = (m + t.log())[..., 0]
        o[h:h + step] = torch.matmul(x, v[h:h + step].contiguous()) / torch.where(t == 0, torch.ones_like(t), t)
    return o.view(H, lq, D).transpose(0, 1).to(torch.bfloat16), z.view(H, lq).t()


def _rotary_plain(c, s):
    axes = s["axes"]
    half = sum(axes) // 2
    axis = torch.tensor([a for a, d in enumerate(axes) for _ in range(d // 2)], device="cuda")
    if c["ladder"] == "axis":
        power = [2 * j / d for d in axes for j in range(d // 2)]
    else:
        power = [i / half for i in range(half)]
    freq = c["theta"] ** -torch.tensor(power, dtype=torch.float64, device="cuda")
    angle = s["positions"].double()[:, axis] * freq
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    out = []
    for n in "qk":
        x = s[n].float()
        if c["norm"]:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * s[n + "_weight"].float()
        if c["pairs"] == "adjacent":
            m, k = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
            y = torch.stack([m * cos - k * sin, m * sin + k * cos], -1).flatten(-2)
        else:
            m, k = x[..., :half], x[..., half:2 * half]
            y = torch.cat([m * cos - k * sin, m * sin + k * cos], -1)
        out.append(torch.cat([y, x[..., 2 * half:]], -1).to(torch.bfloat16))
    return tuple(out)


# ---- the same in 64 bits, from the definitions -------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return _rotary64(case, s) if case["op"] == "rotary" else _attention64(case, s)


def _rotary64(c, s):
    axes, R = s["axes"], sum(s["axes"])
    out = []
    for n in "qk":
        x = s[n].double()
        if c["norm"]:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / c["D"] + 1e-6) * s[n + "_weight"].double()
        y, i = x.clone(), 0
        for a, d in enumerate(axes):
            for j in range(d // 2):
                e = 2.0 * j / d if c["ladder"] == "axis" else 2.0 * i / R
                turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                                   s["positions"][:, a].double() * math.exp(-e * math.log(c["theta"])))
                m, k = (2 * i, 2 * i + 1) if c["pairs"] == "adjacent" else (i, i + R // 2)
                z = torch.complex(x[:, :, m], x[:, :, k]) * turn[:, None]
                y[:, :, m], y[:, :, k] = z.real, z.imag
                i += 1
        out.append(y)
    return tuple(out)


def _attention64(c, s):
    q, k = _lengths(c)
    H, D, P = c["heads"], c["D"], c["prefix"]
    G = H // c["kv_heads"]
    Q, K, V = (s[n].reshape(-1, s[n].shape[-2], D) for n in "qkv")
    out = torch.zeros((sum(q), H, D), dtype=torch.float64, device="cuda")
    lse = torch.full((sum(q), H), -math.inf, dtype=torch.float64, device="cuda")
    for h in range(H):
        i = j = 0
        for lq, lk in zip(q, k):
            k_h, v_h = K[j:j + lk, h // G].double(), V[j:j + lk, h // G].double()
            if P:
                k_h = torch.cat([s["prefix"][0][:, h // G].double(), k_h])
                v_h = torch.cat([s["prefix"][1][:, h // G].double(), v_h])
            for at in range(0, lq if P + lk else 0, 4096):
                rows = slice(i + at, i + min(at + 4096, lq))
                w = (Q[rows, h].double() @ k_h.t().contiguous()) / math.sqrt(D)
                if c["causal"]:
                    first = P + lk - lq + 1 + at  # the first key that the chunk's first query does not see
                    gone = torch.ones_like(w, dtype=torch.bool).triu(first)
                    gone[:, :P] = False
                    w[gone] = -math.inf
                lse[rows, h] = torch.logsumexp(w, 1)
                w = torch.exp(w - lse[rows, h, None])
                out[rows, h] = torch.where(lse[rows, h, None] == -math.inf, torch.zeros_like(w[:, :1]), w @ v_h)
            i, j = i + lq, j + lk
    shape = s["q"].shape
    return (out.view(shape), lse.view(shape[:-1])) if c["lse"] else out.view(shape)
