"""Plain fp64 CPU oracle of the 8-bit linear layer and of the block norms.

TEST INFRASTRUCTURE ONLY, as lynx_oracle.py; it shares no code, table or
constant with the HIP library.  Definitions (include/lynx.h):

  * e4m3: 1 sign bit, 4 exponent bits (bias 7), 3 fraction bits; exponent 0 is
    subnormal; 0x7F / 0xFF are NaN; largest value 448.
  * a block's scale is 2^e, e the smallest integer >= -127 with amax <= 448 * 2^e
    (amax = 0: e = 0; a NaN or an infinity inside: NaN); values are x / 2^e
    rounded to nearest even.
  * blocks: 128 channels of a row (activation), 128 rows x 128 channels (weight).
"""
from __future__ import annotations

import numpy as np

BLOCK = 128
SCALE_NAN = 255


def e4m3_table() -> np.ndarray:
    """The value of each of the 256 codes, from the format's definition."""
    out = np.empty(256)
    for code in range(256):
        sign = -1.0 if code & 0x80 else 1.0
        exp, frac = (code >> 3) & 15, code & 7
        if exp == 15 and frac == 7:
            out[code] = np.nan
        elif exp == 0:
            out[code] = sign * frac / 8 * 2.0 ** -6
        else:
            out[code] = sign * (1 + frac / 8) * 2.0 ** (exp - 7)
    return out


def e4m3_encode(v: np.ndarray) -> np.ndarray:
    """Codes of the e4m3 values nearest to v (|v| <= 448), ties to even."""
    mag = np.abs(v)
    with np.errstate(divide="ignore"):
        exp = np.where(mag > 0, np.floor(np.log2(np.where(mag > 0, mag, 1.0))), -6)
    exp = np.where(np.exp2(exp) > mag, exp - 1, exp)        # log2 rounded up
    exp = np.where(np.exp2(exp + 1) <= mag, exp + 1, exp)   # log2 rounded down
    exp = np.maximum(exp, -6)
    units = np.rint(mag / np.exp2(exp - 3)).astype(np.int64)  # 0 .. 16 eighths; np.rint: ties to even
    over = units == 16
    exp, units = np.where(over, exp + 1, exp), np.where(over, 8, units)
    code = np.where(units < 8, units, (exp.astype(np.int64) + 7) * 8 + units - 8)
    return (code | np.where(np.signbit(v), 0x80, 0)).astype(np.uint8)


def scale_exponent(amax: np.ndarray) -> np.ndarray:
    """e of the definition (finite amax), by search from below on exact powers."""
    amax = np.asarray(amax, dtype=np.float64)
    with np.errstate(divide="ignore"):
        e = np.floor(np.log2(np.where(amax > 0, amax, 1.0) / 448.0)) - 1
    for _ in range(3):
        e = np.where(448.0 * np.exp2(e) < amax, e + 1, e)
    return np.where(amax > 0, np.maximum(e, -127), 0).astype(np.int64)


def _scale_bytes(blocks: np.ndarray) -> np.ndarray:
    """blocks [..., n] -> the scale byte of each."""
    bad = ~np.isfinite(blocks).all(-1)
    amax = np.abs(np.where(bad[..., None], 0.0, blocks)).max(-1)
    return np.where(bad, SCALE_NAN, scale_exponent(amax) + 127).astype(np.uint8)


def _encode_blocks(x: np.ndarray, byte: np.ndarray) -> np.ndarray:
    """Codes of x with the scale byte of every element; 0 where it is NaN."""
    bad = byte == SCALE_NAN
    scaled = np.where(bad, 0.0, x) / np.exp2(np.where(bad, 127, byte).astype(np.float64) - 127)
    return e4m3_encode(scaled)


def quantize(x: np.ndarray):
    """x [M, K] -> codes [M, K], scale bytes [M, ceil(K/128)]."""
    M, K = x.shape
    kb = -(-K // BLOCK)
    byte = np.stack([_scale_bytes(x[:, BLOCK * i:BLOCK * (i + 1)]) for i in range(kb)], 1)
    return _encode_blocks(x, byte.repeat(BLOCK, 1)[:, :K]), byte


def quantize_weight(w: np.ndarray):
    """w [N, K] -> codes [N, K], scale bytes [ceil(N/128), ceil(K/128)]."""
    N, K = w.shape
    byte = np.array([[_scale_bytes(w[r:r + BLOCK, c:c + BLOCK].reshape(-1))
                      for c in range(0, K, BLOCK)] for r in range(0, N, BLOCK)], dtype=np.uint8)
    return _encode_blocks(w, byte.repeat(BLOCK, 0)[:N].repeat(BLOCK, 1)[:, :K]), byte


def stored_scales(byte: np.ndarray) -> np.ndarray:
    """Activation scale bytes [M, blocks] as stored: [ceil(blocks/4), M, 4], 127 elsewhere."""
    M, kb = byte.shape
    full = np.full((M, -(-kb // 4) * 4), 127, dtype=np.uint8)
    full[:, :kb] = byte
    return np.ascontiguousarray(full.reshape(M, -1, 4).transpose(1, 0, 2))


def stored_weight_scales(byte: np.ndarray) -> np.ndarray:
    """Weight scale bytes as stored: rows filled up to a multiple of four with 127."""
    full = np.full((byte.shape[0], -(-byte.shape[1] // 4) * 4), 127, dtype=np.uint8)
    full[:, :byte.shape[1]] = byte
    return full


def values(codes: np.ndarray, byte: np.ndarray, rows_per_scale: int = 1) -> np.ndarray:
    """What an operand stands for: byte one per row (or rows_per_scale rows) and 128 channels."""
    N, K = codes.shape
    s = np.where(byte == SCALE_NAN, np.nan, np.exp2(byte.astype(np.float64) - 127))
    return e4m3_table()[codes] * s.repeat(rows_per_scale, 0)[:N].repeat(BLOCK, 1)[:, :K]


def linear(xv: np.ndarray, wv: np.ndarray):
    """Y = X W^T of the values of two operands, and sum |x w|, the scale of its error."""
    return xv @ wv.T, np.abs(xv) @ np.abs(wv).T


def _norm(v, kind, weight, bias, eps):
    """(result, the magnitudes whose fp32 rounding can show in it)."""
    if kind is None:
        return v, np.abs(v)
    mean = v.mean(1, keepdims=True) if kind == "layer" else 0.0
    t = v - mean
    rs = 1.0 / np.sqrt((t * t).mean(1, keepdims=True) + eps)
    out, mag = t * rs, (np.abs(v) + np.abs(v).mean(1, keepdims=True)) * rs
    if weight is not None:
        out, mag = out * weight, mag * np.abs(weight)
    if bias is not None:
        out, mag = out + bias, mag + np.abs(bias)
    return out, mag


def block_norm(x, y=None, gate=None, post_norm=None, post_weight=None, post_bias=None,
               post_eps=1e-6, residual_scale=1.0, norm=None, weight=None, bias=None, scale=None,
               shift=None, eps=1e-6):
    """x', h of lynx_block_norm, each with the magnitudes of its terms; gate, scale
    and shift [samples, C]."""
    def rows(p):
        return None if p is None else p[np.arange(len(x)) * len(p) // len(x)]

    u, umag = x, np.abs(x)
    if y is not None:
        z, zmag = _norm(y, post_norm, post_weight, post_bias, post_eps)
        g = 1.0 if gate is None else rows(gate)
        u, umag = residual_scale * x + g * z, np.abs(residual_scale * x) + np.abs(g) * zmag
    if norm is None:
        return u, umag, None, None
    # the error of u reaches h as umag / |u| does: its magnitudes take u's place
    h, _ = _norm(u, norm, weight, bias, eps)
    t = u - u.mean(1, keepdims=True) if norm == "layer" else u
    rs = 1.0 / np.sqrt((t * t).mean(1, keepdims=True) + eps)
    # an error d in every u moves rs by at most rms(d) rs^2, and so h by |t| rs more
    hmag = (umag + umag.mean(1, keepdims=True)) * rs
    hmag = hmag + np.abs(t) * rs * rs * np.sqrt((umag ** 2).mean(1, keepdims=True))
    if weight is not None:
        hmag = hmag * np.abs(weight)
    if bias is not None:
        hmag = hmag + np.abs(bias)
    if scale is not None:
        h, hmag = h * (1 + rows(scale)), hmag * (1 + np.abs(rows(scale)))
    if shift is not None:
        h, hmag = h + rows(shift), hmag + np.abs(rows(shift))
    return u, umag, h, hmag
