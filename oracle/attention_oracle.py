"""Plain fp64 CPU oracle of rotary positions and of attention.

TEST INFRASTRUCTURE ONLY, as lynx_oracle.py; it shares no code, table or
constant with the HIP library.  Definitions (include/lynx.h):

  * rotary: axis i of d_i channels turns its pair j by positions[t, i] *
    theta^(-2 j / d_i) ("axis") or, pair p of all R / 2, theta^(-2 p / R)
    ("joint"); a pair is channels (2 p, 2 p + 1) or (p, p + R / 2).
  * attention: query i of Lq sees all prefix keys and own keys j, causal: j <=
    i + Lk - Lq; out = sum p v / sum p, p = exp(scale q.k), 0 where nothing is
    seen; lse = log sum p, -inf there.
"""
from __future__ import annotations

import numpy as np


def rotary(x, positions, axes, theta=10000.0, pairs="adjacent", ladder="axis", norm=False,
           weight=None, eps=1e-6):
    """x [T, H, D], positions [T, len(axes)] -> the turned x, fp64."""
    x = np.array(x, dtype=np.float64)
    D, R = x.shape[-1], sum(axes)
    if norm:
        x = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
        if weight is not None:
            x = x * np.asarray(weight, dtype=np.float64)
    out = x.copy()
    p = 0
    for i, d in enumerate(axes):
        for j in range(d // 2):
            e = j / (d / 2) if ladder == "axis" else p / (R / 2)
            a = np.asarray(positions)[:, i].astype(np.float64) * float(theta) ** -e
            m, n = (2 * p, 2 * p + 1) if pairs == "adjacent" else (p, p + R // 2)
            c, s = np.cos(a)[:, None], np.sin(a)[:, None]
            out[:, :, m] = x[:, :, m] * c - x[:, :, n] * s
            out[:, :, n] = x[:, :, m] * s + x[:, :, n] * c
            p += 1
    assert p == R // 2 and R <= D
    return out


def visible(lq, lk, causal, prefix=0):
    """[lq, prefix + lk] truth values: the keys that a query sees."""
    own = np.ones((lq, lk), dtype=bool)
    if causal:
        own = np.arange(lk)[None, :] <= np.arange(lq)[:, None] + lk - lq
    return np.concatenate([np.ones((lq, prefix), dtype=bool), own], axis=1)


def attention(q, k, v, lens_q, lens_k, causal=False, scale=None, prefix=None):
    """q [Tq, H, D], k and v [Tk, KV, D] packed from token 0 on; prefix: (k, v).

    Returns out [Tq, H, D], lse [Tq, H], and for error bounds dev [Tq, H, D] =
    sqrt(sum p (v - out)^2 / sum p), which is sum p |v - out| / sum p or more; size [Tq, H] =
    the norm over channels of sqrt(sum p^2 (v - out)^2) / sum p; and spread [Tq, H], the largest
    scale * sum |q_d k_d| of a key that is seen.
    """
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    Tq, H, D = q.shape
    G = H // k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    out, dev = np.zeros_like(q), np.zeros_like(q)
    lse, spread, size = np.full((Tq, H), -np.inf), np.zeros((Tq, H)), np.zeros((Tq, H))
    i = j = 0
    for lq, lk in zip(lens_q, lens_k):
        for h in range(H):
            ks, vs = k[j:j + lk, h // G], v[j:j + lk, h // G]
            P = 0
            if prefix is not None:
                P = prefix[0].shape[0]
                ks = np.concatenate([np.asarray(prefix[0][:, h // G], dtype=np.float64), ks])
                vs = np.concatenate([np.asarray(prefix[1][:, h // G], dtype=np.float64), vs])
            see = visible(lq, lk, causal, P)
            rows = np.flatnonzero(see.any(axis=1))
            if rows.size == 0:
                continue
            s = np.where(see[rows], scale * (q[i + rows, h] @ ks.T), -np.inf)
            top = s.max(axis=1, keepdims=True)
            p = np.exp(s - top)
            l = p.sum(axis=1, keepdims=True)
            out[i + rows, h] = p @ vs / l
            o = out[i + rows, h]
            dev[i + rows, h] = np.sqrt(np.maximum(p @ vs ** 2 / l - o ** 2, 0))
            p2 = (p / l) ** 2
            size[i + rows, h] = np.sqrt(np.maximum(
                (p2 @ vs ** 2 - 2 * o * (p2 @ vs) + o ** 2 * p2.sum(axis=1, keepdims=True)).sum(axis=1), 0))
            lse[i + rows, h] = (top + np.log(l))[:, 0]
            a = scale * (np.abs(q[i + rows, h]) @ np.abs(ks.T))
            spread[i + rows, h] = np.where(see[rows], a, 0).max(axis=1)
        i, j = i + lq, j + lk
    return out, lse, dev, size, spread
