"""Plain fp64 oracle of the attention operators (include/gdn_attn.h) in numpy: one
sequence, one head after the other, no code shared with the HIP path.

Each function returns its results with a bound on what an fp32 evaluation may be off
by, derived from the same inputs (U = 2^-24, half an ulp of 1 in fp32).  The bounds count
roundings; nothing in them is fitted.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24
HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
LEAST = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}  # half the smallest step


def rounded(ref, err, dtype):
    """`err` and one rounding to the stored type."""
    h = HALF_STEP[dtype]
    return err * (1 + h) + h * np.abs(ref) + LEAST[dtype]


def positions(cu, kv_len):
    """(sequence, position) of each token."""
    seq = np.repeat(np.arange(len(cu) - 1), np.diff(cu))
    t = np.arange(len(seq)) - np.asarray(cu)[seq]
    return seq, np.asarray(kv_len)[seq] - np.diff(cu)[seq] + t


def rotated(x, P, freq, pairs, weight=None, eps=1e-6, scale=1.0):
    """(result, bound) of rows [T][heads][D] at the positions P.

    Norm: D squares summed in any order lose at most (D + 2) U of their sum, half of it
    after the root; root, quotient and two products 5 U.  Cosine and sine: the turns enter
    them rounded (pi U), the function 4 U, the factor and its product U each: 10 U; the
    64-bit angle 2^-51 of itself.  Each pair's two products and their sum 3 U."""
    D, r = x.shape[-1], 2 * len(freq)
    err = np.zeros_like(x)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
        err = ((D + 2) / 2 + 5) * U * np.abs(x)
    angle = P[:, None] * freq
    c, s = scale * np.cos(angle)[:, None], scale * np.sin(angle)[:, None]
    de = scale * (10 * U + 2.0 ** -51 * np.abs(angle)[:, None])
    a, b = (np.arange(0, r, 2), np.arange(1, r, 2)) if pairs else (np.arange(r // 2), np.arange(r // 2, r))
    y, e = x.copy(), err.copy()
    xa, xb, ea, eb = x[..., a], x[..., b], err[..., a], err[..., b]
    y[..., a], y[..., b] = xa * c - xb * s, xb * c + xa * s
    off = (np.abs(xa) + np.abs(xb)) * (de + 3 * U * scale) + (ea + eb) * scale
    e[..., a], e[..., b] = off, off
    return y, e


def keys_of(cache, table, n, h, length, page):
    """Rows [length][D] of head h of sequence n; cache [pages][KV][page][D]."""
    at = np.arange(length)
    return cache[table[n, at // page], h, at % page]


def attention(cu, kv_len, table, q, k_cache, v_cache, page, scale, window=0, gate=None, weight_step=0.0, weight_least=0.0):
    """(out, bound) [T][H][D].

    A score loses (D + 2) U of its absolute products, the exponent's argument 4 U of the
    score and of the largest one, exp and its factor 4 U: a weight is off by e_j of
    itself, o by sum w_j e_j |V_j - o|.  Sums over keys run in blocks of 64 at most, and the
    blocks' one after the other (or in parts that are joined): (64 + keys / 32 + 16) U of the
    absolute terms, and as much of the sum of weights.  weight_step, weight_least: the weights as operands of the
    product with V are off by that much of themselves, and at least of the largest weight.  The gate's
    sigmoid loses (4 + |gate|) U."""
    T, H, D = q.shape
    KV = k_cache.shape[1]
    out, err = np.zeros((T, H, D)), np.zeros((T, H, D))
    for n in range(len(cu) - 1):
        new, L = cu[n + 1] - cu[n], kv_len[n]
        if new == 0:
            continue
        p = L - new + np.arange(new)
        j = np.arange(L)
        seen = j <= p[:, None]
        if window:
            seen &= j > p[:, None] - window
        for h in range(H):
            K, V = (keys_of(c, table, n, h * KV // H, L, page) for c in (k_cache, v_cache))
            x = q[cu[n]:cu[n + 1], h]
            any_ = seen.any(1)
            used = seen.any(0)
            K, V = np.where(used[:, None], K, 0.0), np.where(used[:, None], V, 0.0)
            s = np.where(seen, scale * (x @ K.T), -np.inf)
            m = np.where(any_, s.max(1, initial=-np.inf), 0.0)[:, None]
            w = np.exp(s - m)
            l = np.where(any_, w.sum(1), 1.0)[:, None]
            wn = w / l
            o = wn @ V
            fin = np.where(seen, s, 0.0)
            e = np.where(seen, scale * (D + 2) * U * (np.abs(x) @ np.abs(K).T) + 4 * U * (np.abs(fin) + np.abs(m)) + 4 * U, 0.0)
            e = e + e.max(1, initial=0.0, keepdims=True)  # the largest score's own error
            steps = (64 + seen.sum(1, keepdims=True) / 32 + 16) * U
            mag = wn @ np.abs(V)
            off = (wn * e) @ np.abs(V) + (wn * e).sum(1, keepdims=True) * np.abs(o) + 2 * steps * mag
            off += weight_step * mag + weight_least * (seen @ np.abs(V)) / l
            out[cu[n]:cu[n + 1], h], err[cu[n]:cu[n + 1], h] = o, off
    if gate is not None:
        sig = 1 / (1 + np.exp(-gate))
        err = err * sig + np.abs(out) * sig * (4 + np.abs(gate)) * U * 2
        out = out * sig
    return out, err
