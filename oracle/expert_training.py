"""What training the experts adds to an MoE layer, in float64: the gradient of the
experts' weights, MXFP4 quantisation of the weights and back, the root-mean-square
norm in front of the layer with its gradient, 8-bit rows into expert order.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).

Values are float64, formats are decoded exactly, and nothing is rounded except
where a result is stated as codes or as BF16.
"""
from __future__ import annotations

import numpy as np

from .formats import E8M0_TABLE, bf16_bits_to_f64, decode_e2m1_packed, round_f64_to_bf16_bits
from .moe_io import e4m3_rne, scale_exponent

W_GROUP, A_GROUP = 32, 128
_E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


# ------------------------------------------------- gradient of the weights --

def wgrad(dy, x, offsets, dw_init=None):
    """dw[e] = dw_init[e] + dy[off[e]:off[e+1]]^T x[...], and the terms' magnitudes' sum.
    Experts whose offsets are not monotone or leave the rows have no rows."""
    E, rows = len(offsets) - 1, dy.shape[0]
    dw = np.zeros((E, dy.shape[1], x.shape[1])) if dw_init is None else np.array(dw_init)
    mag = np.abs(dw)
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if 0 <= lo <= hi <= rows:
            dw[e] += dy[lo:hi].T @ x[lo:hi]
            mag[e] += np.abs(dy[lo:hi]).T @ np.abs(x[lo:hi])
    return dw, mag


# ---------------------------------------------------------- 4-bit weights --

def weight_exponent(amax):
    """Smallest integer e with amax <= 6 * 2^e; 0 for amax == 0; clamped to [-127, 127]."""
    if amax == 0.0:
        return 0
    e = int(np.floor(np.log2(amax / 6.0)))
    while amax > 6.0 * 2.0 ** e:
        e += 1
    while amax <= 6.0 * 2.0 ** (e - 1):
        e -= 1
    return max(-127, min(127, e))


def e2m1_rne(q):
    """E2M1 codes of values |q| <= 6, round to nearest, ties to the even code."""
    mag = np.abs(q)
    near = np.abs(mag[..., None] - _E2M1)
    best = near.min(-1, keepdims=True)
    tied = near == best                                   # one code, or two neighbours
    code = tied.argmax(-1)
    code = np.where((tied.sum(-1) == 2) & (code % 2 == 1), code + 1, code)
    return (code | np.where(np.signbit(q), 8, 0)).astype(np.uint8)


def quantize_weights(w):
    """[..., N, K] -> (packed E2M1 codes [..., N, K/2], E8M0 codes [..., N, K/32])."""
    w = np.asarray(w, dtype=np.float64)
    g = w.reshape(-1, W_GROUP)
    codes = np.zeros(g.shape, dtype=np.uint8)
    scales = np.empty(g.shape[0], dtype=np.uint8)
    for i, v in enumerate(g):
        if not np.isfinite(v).all():
            scales[i] = 255
            continue
        e = weight_exponent(float(np.abs(v).max()))
        scales[i] = 127 + e
        codes[i] = e2m1_rne(v / 2.0 ** e)
    codes = codes.reshape(w.shape)
    packed = codes[..., 0::2] | (codes[..., 1::2] << 4)
    return packed, scales.reshape(*w.shape[:-1], w.shape[-1] // W_GROUP)


def dequantize_weights(packed, scales):
    """The numbers of packed E2M1 codes with their scales (code 255: NaN)."""
    s = np.repeat(E8M0_TABLE[np.asarray(scales)], W_GROUP, axis=-1)
    return decode_e2m1_packed(packed) * s


# ------------------------------------------------------------------- norm --

def rmsnorm(x, residual, gain, eps):
    """(s, r, v): s = bf16(x + residual) (x without one), r = 1/rms, v = s r gain."""
    s = x
    if residual is not None:
        s = bf16_bits_to_f64(round_f64_to_bf16_bits(x + residual))
    with np.errstate(invalid="ignore"):
        r = 1.0 / np.sqrt((s * s).mean(axis=1) + eps)
        return s, r, s * r[:, None] * gain


def quantize_rows_f64(v):
    """E4M3 codes and E8M0 codes of [M, D] numbers by the activations' rule."""
    M, D = v.shape
    g = v.reshape(-1, A_GROUP)
    codes = np.empty(g.shape, dtype=np.uint8)
    scales = np.empty(g.shape[0], dtype=np.uint8)
    for i, u in enumerate(g):
        if not np.isfinite(u).all():
            scales[i], codes[i] = 0xFF, 0x7F
            continue
        e = scale_exponent(float(np.abs(u).max()))
        scales[i] = 127 + e
        codes[i] = e4m3_rne(u / 2.0 ** e)
    return codes.reshape(M, D), scales.reshape(M, D // A_GROUP)


def rmsnorm_bwd(dy, s, gain, r, dsum=None):
    """(dx, dgain) and the magnitudes' sums of their terms."""
    D = s.shape[1]
    n, u = s * r[:, None], dy * gain * r[:, None]
    mean = (u * n).sum(1, keepdims=True) / D
    dx = u - n * mean
    mag = np.abs(u) + np.abs(n) * (np.abs(u * n).sum(1, keepdims=True) / D)
    if dsum is not None:
        dx, mag = dx + dsum, mag + np.abs(dsum)
    return dx, (dy * n).sum(0), mag, np.abs(dy * n).sum(0)


# ------------------------------------------------------------ 8-bit rows --

def dispatch_acts(a, scale, place, rows_init, scale_init):
    """Codes and scales of token t to the rows place[t, j]; the other rows as they were."""
    rows, scales = np.array(rows_init), np.array(scale_init)
    for t, j in zip(*np.nonzero((place >= 0) & (place < rows.shape[0]))):
        rows[place[t, j]], scales[place[t, j]] = a[t], scale[t]
    return rows, scales
