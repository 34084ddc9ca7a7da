"""CPU oracle (numpy, fp64) of the attention half of a decoder layer: position
rotation with the optional per-head RMS norm, append to a paged cache, and
causal attention over it.  Inputs are the bf16 values the library reads (as
floats); outputs are unrounded, with bounds on what the library's arithmetic
may add.

Roundings the bounds count: one to bf16 at the end (relative error at most
2^-8, half a bf16 step), the softmax weights to bf16 before the value product
(2^-8 each), and fp32 steps of 2^-24.
"""
from __future__ import annotations

import math
from typing import List, Optional, Tuple

import numpy as np

U16 = 2.0 ** -8    # half a bf16 step, relative
U32 = 2.0 ** -24   # half an fp32 step, relative


def frequencies(rot: int, theta: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                original_len: float = 8192.0, low: float = 1.0, high: float = 4.0) -> np.ndarray:
    """Radians per position of the rot / 2 pairs."""
    f = np.array([theta ** (-2.0 * i / rot) for i in range(rot // 2)])
    if scaling == "linear":
        return f / factor
    if scaling == "by_parts":
        w = np.clip((original_len * f / (2.0 * math.pi) - low) / (high - low), 0.0, 1.0)
        return (1.0 - w) * f / factor + w * f
    assert scaling == "none"
    return f


def rms_norm(x: np.ndarray, w: np.ndarray, eps: float) -> np.ndarray:
    x = x.astype(np.float64)
    return x * w.astype(np.float64) / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)


def rotate(x: np.ndarray, pos: np.ndarray, freq: np.ndarray, layout: str = "half",
           amplitude: float = 1.0) -> Tuple[np.ndarray, np.ndarray]:
    """x: T x heads x D at positions pos: T.  Returns the rotated rows and the
    per-element magnitude |x1| + |x2| (|x| where nothing turns) that fp32
    errors scale with."""
    x = x.astype(np.float64)
    half = len(freq)
    ang = pos.astype(np.float64)[:, None] * freq[None, :]
    c, s = amplitude * np.cos(ang)[:, None, :], amplitude * np.sin(ang)[:, None, :]
    y, mag = x.copy(), np.abs(x)
    if layout == "half":
        i1, i2 = slice(0, half), slice(half, 2 * half)
    else:
        i1, i2 = slice(0, 2 * half, 2), slice(1, 2 * half, 2)
    y[..., i1] = x[..., i1] * c - x[..., i2] * s
    y[..., i2] = x[..., i1] * s + x[..., i2] * c
    m = amplitude * (np.abs(x[..., i1]) + np.abs(x[..., i2]))
    mag[..., i1] = m
    mag[..., i2] = m
    return y, mag


def rotate_bound(y: np.ndarray, mag: np.ndarray, normed: bool) -> np.ndarray:
    """bf16 rounding of the result, plus fp32: the remainder of the angle
    (2 pi 2^-25), sine, cosine and amplitude (4 steps), two products and a sum;
    with a norm the sum of squares (at most 16 sums per thread and 3 levels),
    root, division and products, 32 steps in all."""
    return U16 * np.abs(y) + (1 + U16) * (16 + (32 if normed else 0)) * U32 * mag + 1e-38


def rows(cu_q, kv_len):
    """[(row, sequence, position), ...] of the rows that hold tokens."""
    out = []
    for b in range(len(kv_len)):
        for t in range(int(cu_q[b]), int(cu_q[b + 1])):
            p = int(kv_len[b]) - (int(cu_q[b + 1]) - t)
            if p >= 0:
                out.append((t, b, p))
    return out


def append(cacheK: np.ndarray, cacheV: np.ndarray, k: np.ndarray, v: np.ndarray, cu_q, kv_len, table) -> List[tuple]:
    """Writes rows into the caches (n_pages x heads x page x D); returns the
    (row, page, slot) triples written."""
    P = cacheK.shape[2]
    done = []
    for t, b, p in rows(cu_q, kv_len):
        if p // P >= table.shape[1] or not 0 <= table[b, p // P] < cacheK.shape[0]:
            continue
        pg = table[b, p // P]
        cacheK[pg, :, p % P] = k[t]
        cacheV[pg, :, p % P] = v[t]
        done.append((t, int(pg), p % P))
    return done


def gather(cache: np.ndarray, table_row, n: int) -> np.ndarray:
    """Keys or values of n positions: n x heads x D; zeros where the page is
    not in the cache."""
    n_pages, H, P, D = cache.shape
    out = np.zeros((n, H, D), np.float64)
    for j0 in range(0, n, P):
        pg = int(table_row[j0 // P])
        m = min(P, n - j0)
        if 0 <= pg < n_pages:
            out[j0:j0 + m] = cache[pg, :, :m].transpose(1, 0, 2)
    return out


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, limit: np.ndarray,
           scale: float) -> Tuple[np.ndarray, np.ndarray]:
    """q: n x Hq x D, k, v: m x Hkv x D; row i sees keys [0, limit[i]).
    Returns o and a bound on the library's distance from it."""
    n, Hq, D = q.shape
    m, Hkv, _ = k.shape
    g = Hq // Hkv
    o = np.zeros((n, Hq, D))
    tol = np.zeros((n, Hq, D))
    seen = np.arange(m)[None, :] < limit[:, None]
    for h in range(Hq):
        kh, vh, qh = k[:, h // g], v[:, h // g], q[:, h].astype(np.float64)
        with np.errstate(invalid="ignore"):
            s = scale * (qh @ kh.T)
        s = np.where(seen, s, -np.inf)
        top = np.max(s, axis=1, keepdims=True, initial=-np.inf)
        w = np.where(seen, np.exp(s - np.where(np.isfinite(top), top, 0.0)), 0.0)
        z = w.sum(1, keepdims=True)
        w = np.divide(w, z, out=np.zeros_like(w), where=z > 0)
        o[:, h] = w @ vh
        wv = w @ np.abs(vh)
        # an fp32 score: D products summed in any order, then scale and log2 e;
        # the exponential of it: 2^-22 by the hardware's, 2.9e-6 (49 steps) by a
        # degree-4 polynomial; the sum over the row's keys in any order
        mag = np.where(seen, abs(scale) * (np.abs(qh) @ np.abs(kh).T), 0.0)
        ds = (D + 8) * U32 * np.max(mag, axis=1, initial=0.0)[:, None]
        tol[:, h] = U16 * np.abs(o[:, h]) + wv * (1 + U16) * (U16 + 4 * ds + (limit[:, None].clip(0) + 64) * U32)
    return o, tol + 1e-38


def attention(q: np.ndarray, cacheK: np.ndarray, cacheV: np.ndarray, cu_q, kv_len, table,
              scale: Optional[float] = None) -> Tuple[np.ndarray, np.ndarray, np.ndarray]:
    """q: T x Hq x D.  Returns o, its bound, and which rows are written."""
    T, Hq, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    o, tol = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    written = np.zeros(T, bool)
    P = cacheK.shape[2]
    for b in range(len(kv_len)):
        r0, r1 = int(cu_q[b]), int(cu_q[b + 1])
        if r1 == r0:
            continue
        written[r0:r1] = True
        kv = min(int(kv_len[b]), table.shape[1] * P)
        pos = int(kv_len[b]) - (r1 - np.arange(r0, r1))
        k, v = gather(cacheK, table[b], kv), gather(cacheV, table[b], kv)
        o[r0:r1], tol[r0:r1] = attend(q[r0:r1], k, v, np.minimum(pos + 1, kv), scale)
    return o, tol, written
