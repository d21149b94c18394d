"""Oracle of the paged-cache operators: plain numpy float64, test
infrastructure only.

Definitions (include/kvpop.h states the same ones):
  heads   y = x / sqrt(mean(x^2) + eps) * w; the pairs (a, b) of the first
          rot_dim elements become (a cos - b sin, b cos + a sin) with the
          angle position * inv_freq[i]
  held    e4m3 with one fp32 scale per row: scale = max|x| * c with
          c = 1 / 448 rounded to fp32 (formed in fp32), held value = e4m3(x / scale), the quotient rounded to fp32
          first (for bf16 rows it often falls on the middle between two e4m3
          values, so its rounding is part of the definition); rows whose scale is below the
          smallest normal fp32 number are held as zeros; rows with an
          infinity or a NaN read back as NaN
  attend  s_j = scale q . k_j, capped: c tanh(s_j / c); out = softmax(s) v
          over the attended tokens, lse = log sum e^s; no token: 0 and -inf
"""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0


def heads(x, weight, eps, positions, inv_freq, rot_scale=1.0, interleaved=False):
    """x [tokens][heads][d], positions [tokens], weight [d] or None, inv_freq [rot_dim / 2]."""
    x = np.asarray(x, np.float64).copy()
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    half = len(inv_freq)
    angle = np.asarray(positions, np.float64)[:, None] * np.asarray(inv_freq, np.float64)[None, :]
    c, s = (rot_scale * f(angle)[:, None, :] for f in (np.cos, np.sin))
    ia, ib = (np.arange(half) * 2, np.arange(half) * 2 + 1) if interleaved else (np.arange(half), np.arange(half) + half)
    a, b = x[..., ia], x[..., ib]
    x[..., ia], x[..., ib] = a * c - b * s, b * c + a * s
    return x


def e4m3_grid():
    """Every non-negative finite e4m3 value, ascending: code c has exponent
    field c >> 3 and fraction c & 7 (fraction / 8 * 2^-6 where the field is 0)."""
    return np.array([(c & 7) / 8 * 2.0 ** -6 if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7) for c in range(127)])


def round_e4m3(x):
    """To the nearest e4m3 value, ties to the even code, beyond 448 to 448."""
    g = e4m3_grid()
    a = np.minimum(np.abs(x), E4M3_MAX)
    hi = np.searchsorted(g, a).clip(1, 126)
    lo = hi - 1
    mid = (g[lo] + g[hi]) / 2
    up = (a > mid) | ((a == mid) & (hi % 2 == 0))
    return np.copysign(np.where(up, g[hi], g[lo]), x)


def hold_e4m3(x):
    """Rows x [..., d] (exact in fp32) -> held values and scales, float64."""
    x = np.asarray(x, np.float64)
    top = np.abs(x).max(-1)
    with np.errstate(all="ignore"):
        scale = top.astype(np.float32) * (np.float32(1) / np.float32(E4M3_MAX))
        scale = np.where(np.isfinite(scale), np.where(scale < np.finfo(np.float32).tiny, np.float32(0), scale), np.float32(np.nan))
        s = scale.astype(np.float64)
        ratio = np.where(scale[..., None] > 0, x.astype(np.float32) / scale[..., None], np.float32(0)).astype(np.float64)
    return np.where(np.isnan(s)[..., None], np.nan, round_e4m3(np.nan_to_num(ratio))), s


def attend(q, k, v, scale=None, softcap=0.0, window=0):
    """q [Hq][d], k and v [n][Hkv][d] of one sequence -> out [Hq][d], lse [Hq]."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    n, hkv, d = k.shape
    hq = q.shape[0]
    if window and n > window:
        k, v = k[n - window:], v[n - window:]
    if n == 0:
        return np.zeros((hq, d)), np.full(hq, -np.inf)
    scale = d ** -0.5 if scale is None else scale
    g = hq // hkv
    with np.errstate(all="ignore"):
        s = np.einsum("hgd,nhd->hgn", q.reshape(hkv, g, d), k) * scale
        if softcap:
            s = softcap * np.tanh(s / softcap)
        m = s.max(-1, keepdims=True)
        e = np.exp(s - m)
        z = e.sum(-1, keepdims=True)
        out = np.einsum("hgn,nhd->hgd", e, v) / z
        lse = (m + np.log(z))[..., 0]
    return out.reshape(hq, d), lse.reshape(hq)


def attend_slack(q, k, v, scale=None, window=0):
    """How far an fp32 computation of `attend` may be off, element by element,
    before its output is rounded, and its lse.

    A dot product of d terms in fp32 is off by at most (d + 2) u sum|q_i k_i|,
    u = 2^-24; a score off by t scales its weight by e^t, so weights (and their
    sum) are off by 2 t relative.  Weights themselves carry 2^-16 (a weight is
    held as two bf16 terms of 8 bits each), exp2 4 u, and the sums over n
    tokens (n + 64) u relative to sum p |v|."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    n, hkv, d = k.shape
    hq = q.shape[0]
    if window and n > window:
        k, v = k[n - window:], v[n - window:]
    if n == 0:
        return np.zeros((hq, d)), np.zeros(hq)
    scale = d ** -0.5 if scale is None else scale
    u = 2.0 ** -24
    qh = q.reshape(hkv, hq // hkv, d)
    t = (d + 8) * u * (np.einsum("hgd,nhd->hgn", np.abs(qh), np.abs(k)) * scale).max(-1)
    s = np.einsum("hgd,nhd->hgn", qh, k) * scale
    e = np.exp(s - s.max(-1, keepdims=True))
    e /= e.sum(-1, keepdims=True)
    a = np.einsum("hgn,nhd->hgd", e, np.abs(v))
    rel = 4 * t + 2.0 ** -16 + (2 * k.shape[0] + 128) * u
    return (rel[..., None] * a).reshape(hq, d), (t + (2 * k.shape[0] + 128) * u + 8 * u * np.abs(s).max(-1)).reshape(hq)
