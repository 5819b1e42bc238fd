"""The steps of an MoE layer around its GEMMs, in float64: dispatch and combine
with their gradients, SwiGLU with an 8-bit checkpoint, the few-token expert
product, and the router's gate.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).

Every function takes and returns float64 values (formats are decoded by the
caller or here, exactly) and rounds nothing, except where a result is stated
as codes.  ``place[t, j]`` is the sorted row of choice j of token t, entries
outside [0, M*k) take no part.
"""
from __future__ import annotations

import numpy as np

from .formats import E4M3_TABLE, E8M0_TABLE, decode_e2m1_packed
from .moe_io import e4m3_rne

GROUP = 128


# ------------------------------------------------- tokens by expert -------

def _valid(place, rows):
    place = np.asarray(place, dtype=np.int64)
    return place, (place >= 0) & (place < rows)


def dispatch(x, place, weights, rows_init):
    """rows[place[t, j]] = w[t, j] * x[t]; the other rows as in rows_init."""
    rows = np.array(rows_init, dtype=np.float64)
    place, ok = _valid(place, rows.shape[0])
    for t, j in zip(*np.nonzero(ok)):
        rows[place[t, j]] = x[t] if weights is None else weights[t, j] * x[t]
    return rows


def combine(y, place, weights):
    """out[t] = sum_j w[t, j] * y[place[t, j]], and the sum of the terms' magnitudes."""
    place, ok = _valid(place, y.shape[0])
    M, k = place.shape
    w = np.ones((M, k)) if weights is None else weights
    out = np.zeros((M, y.shape[1]))
    mag = np.zeros_like(out)
    for j in range(k):
        at = ok[:, j]
        term = w[at, j:j + 1] * y[place[at, j]]
        out[at] += term
        mag[at] += np.abs(term)
    return out, mag


def row_dots(rows, token, place):
    """<rows[place[t, j]], token[t]> (0 where there is no row), and the sum of magnitudes."""
    place, ok = _valid(place, rows.shape[0])
    dots, mag = np.zeros(place.shape), np.zeros(place.shape)
    for t, j in zip(*np.nonzero(ok)):
        p = rows[place[t, j]] * token[t]
        dots[t, j] = p.sum()
        mag[t, j] = np.abs(p).sum()
    return dots, mag


# --------------------------------------------------------- SwiGLU ---------

def sigmoid(g):
    e = np.exp(-np.abs(g))
    return np.where(g >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def swiglu(z):
    g, u = np.split(np.asarray(z, dtype=np.float64), 2, axis=1)
    return g * sigmoid(g) * u


def swiglu_bwd(dh, z):
    g, u = np.split(np.asarray(z, dtype=np.float64), 2, axis=1)
    s = sigmoid(g)
    return np.concatenate([dh * u * (s + g * s * sigmoid(-g)), dh * g * s], axis=1)


def group_exponents(x):
    """Per 128 elements of a row: smallest e with amax <= 448 * 2^e (0 for amax = 0),
    in [-127, 127]."""
    R, K = x.shape
    amax = np.abs(x).reshape(R, K // GROUP, GROUP).max(axis=-1)
    m, p = np.frexp(amax)                                  # amax = m * 2^p, m in [0.5, 1)
    e = p - 9 + (m > 0.875)                                # 448 = 0.875 * 2^9
    return np.clip(np.where(amax > 0, e, 0), -127, 127), amax


def quantize(x):
    """float64 [R, K] (finite) -> (E4M3 codes, E8M0 codes of 128-element groups)."""
    R, K = x.shape
    e, _ = group_exponents(x)
    q = np.ldexp(x.reshape(R, K // GROUP, GROUP), -e[..., None])
    return e4m3_rne(q).reshape(R, K), (e + 127).astype(np.uint8)


def dequantize(codes, scales):
    R, K = codes.shape
    v = E4M3_TABLE[codes].reshape(R, K // GROUP, GROUP) * E8M0_TABLE[scales][..., None]
    return v.reshape(R, K)


# ------------------------------------------------ few-token experts -------

def expert_matvec(x, ids, w_fp4, w_scale):
    """y[s] = W[ids[s]] x[row(s)] and the sums of the terms' magnitudes; zeros for an id
    outside [0, E).  x: [M, K] or [M*k, K]; ids: [M, k]."""
    E, N, _ = w_fp4.shape
    flat = np.asarray(ids, dtype=np.int64).reshape(-1)
    per_row = flat.size // x.shape[0]
    y, mag = np.zeros((flat.size, N)), np.zeros((flat.size, N))
    for e in np.unique(flat):
        if not 0 <= e < E:
            continue
        w = decode_e2m1_packed(w_fp4[e]) * np.repeat(E8M0_TABLE[w_scale[e]], 32, axis=1)
        at = np.nonzero(flat == e)[0]
        y[at] = x[at // per_row] @ w.T
        mag[at] = np.abs(x[at // per_row]) @ np.abs(w.T)
    return y, mag


# ------------------------------------------------------------ router ------

def router_topk(logits, top_k, renormalize):
    """(ids, weights) of float64 logits [M, E] without NaN or +inf."""
    M, E = logits.shape
    ids = np.full((M, top_k), -1, dtype=np.int32)
    weights = np.zeros((M, top_k))
    for t in range(M):
        l = logits[t]
        if not np.any(l > -np.inf):
            continue
        p = np.exp(l - l.max())
        p /= p.sum()
        order = [e for e in np.argsort(-l, kind="stable") if l[e] > -np.inf][:top_k]
        ids[t, :len(order)] = order
        w = p[order]
        weights[t, :len(order)] = w / w.sum() if renormalize else w
    return ids, weights


def router_value(logits, ids, dweights, renormalize):
    """sum_j w[t, j] * dweights[t, j] per token with the choice held at ids: the scalar whose
    gradient router_topk_bwd is."""
    M, k = ids.shape
    v = np.zeros(M)
    for t in range(M):
        chosen = [j for j in range(k) if ids[t, j] >= 0]
        if not chosen:
            continue
        p = np.exp(logits[t] - logits[t].max())
        p /= p.sum()
        w = p[ids[t, chosen]]
        if renormalize:
            w = w / w.sum()
        v[t] = np.dot(w, dweights[t, chosen])
    return v


def router_topk_bwd(logits, ids, dweights, renormalize):
    M, E = logits.shape
    d = np.zeros((M, E))
    for t in range(M):
        chosen = [j for j in range(ids.shape[1]) if ids[t, j] >= 0]
        if not chosen:
            continue
        at = ids[t, chosen]
        dw = dweights[t, chosen]
        p = np.exp(logits[t] - logits[t].max())
        p /= p.sum()
        if renormalize:
            w = p[at] / p[at].sum()
            d[t, at] = w * (dw - np.dot(w, dw))
        else:
            d[t] = -p * np.dot(p[at], dw)
            d[t, at] += p[at] * dw
    return d
