"""Plain fp64 oracle of the state space layer (include/gdn_ssm.h) in numpy: one
row, one token after the other, no code shared with the HIP path.

Each function returns its results with a bound on what an fp32 evaluation may
be off by, derived from the same inputs (U = 2^-24, half an ulp of 1 in fp32).
The bounds count roundings; nothing in them is fitted.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24
HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def silu(x):
    return x / (1.0 + np.exp(-x))


def _silu_err(pre, pre_err):
    """SiLU's slope is below 1.1; x rcp(1 + exp2(x log2 e)) in fp32 loses |x| U in
    the exponent's rounding, 2 U in exp2, U in the sum, 2 U in rcp, U in the
    product; doubled for second orders."""
    return 1.1 * pre_err + 2 * (6 + np.abs(pre)) * U * np.abs(silu(pre))


def conv(cu, xbc, w, b, hist):
    """(out, bound, new history) of float64 arrays; hist [n][K-1][C]."""
    K = w.shape[1]
    out, err = np.zeros_like(xbc), np.zeros_like(xbc)
    new = np.zeros_like(hist)
    for n in range(len(cu) - 1):
        X = np.concatenate([hist[n], xbc[cu[n]:cu[n + 1]]])
        T = cu[n + 1] - cu[n]
        pre = np.broadcast_to(b, (T, xbc.shape[1])).copy()
        mag = np.abs(pre)
        for k in range(K):
            pre += w[:, k] * X[k:k + T]
            mag += np.abs(w[:, k] * X[k:k + T])
        out[cu[n]:cu[n + 1]] = silu(pre)
        err[cu[n]:cu[n + 1]] = _silu_err(pre, (K + 1) * U * mag)
        new[n] = X[T:]
    return out, err, new


def step_size(raw, dt_bias, A_log, dt_min=0.0, dt_max=np.inf):
    u = raw + dt_bias
    dt = np.clip(np.maximum(u, 0) + np.log1p(np.exp(-np.abs(u))), dt_min, dt_max)
    return dt, -np.exp(A_log) * dt


def scan(cu, xbc, dt, lam, D, state, H, P, G, N, xbc_err=None):
    """(y, y bound, state, state bound).  The bound E of the state follows its own
    recurrence on absolute values: a step's decay is off by at most 8 U of its
    log (softplus, exp(A_log), the product) and 2 U (exp), its written part by 8 U
    (dt, two products), and the sum by U or, in parts of operands, a few U:
    E <- a E + U (16 + 10 |lam|) Sabs, Sabs the state of absolute values."""
    T = xbc.shape[0]
    y, ye = np.zeros((T, H, P)), np.zeros((T, H, P))
    S1, E1 = state.copy(), np.zeros_like(state)
    hg = H // G
    grp = np.arange(H) // hg
    for n in range(len(cu) - 1):
        S, Sa, E = state[n].copy(), np.abs(state[n]), np.zeros_like(state[n])
        for t in range(cu[n], cu[n + 1]):
            row = xbc[t]
            x = row[:H * P].reshape(H, P)
            B = row[H * P:H * P + G * N].reshape(G, N)[grp]
            C = row[H * P + G * N:].reshape(G, N)[grp]
            a = np.exp(lam[t])[:, None, None]
            w = dt[t][:, None, None] * x[:, :, None] * B[:, None, :]
            S = a * S + w
            Sa = a * Sa + np.abs(w)
            E = a * E + U * (16 + 10 * np.abs(lam[t]))[:, None, None] * Sa
            if xbc_err is not None:
                e = xbc_err[t]
                ex = e[:H * P].reshape(H, P)
                eB = e[H * P:H * P + G * N].reshape(G, N)[grp]
                eC = e[H * P + G * N:].reshape(G, N)[grp]
                E += dt[t][:, None, None] * (ex[:, :, None] * np.abs(B)[:, None, :] + (np.abs(x) + ex)[:, :, None] * eB[:, None, :])
            y[t] = (S * C[:, None, :]).sum(-1) + D[:, None] * x
            mag = (Sa * np.abs(C)[:, None, :]).sum(-1) + np.abs(D[:, None] * x)
            ye[t] = (E * np.abs(C)[:, None, :]).sum(-1) + (N + 2) * U * mag
            if xbc_err is not None:
                ye[t] += (Sa * eC[:, None, :]).sum(-1) + np.abs(D)[:, None] * ex
        S1[n], E1[n] = S, E
    return y, ye, S1, E1


def scan_magnitude(cu, xbc, dt, lam, D, state, H, P, G, N):
    """y of the absolute values: what a relative error of an operand scales with."""
    return scan(cu, np.abs(xbc), dt, lam, np.abs(D), np.abs(state), H, P, G, N)[0]


def group_norm(x, z, w, b, groups, eps, centre, last):
    """(y, bound); z, w, b may be None.  A sum over n values loses at most 80 U of
    the sum of absolute values (64 in a lane, then a tree)."""
    rows, ch = x.shape
    sig = np.ones_like(x) if z is None else silu(z)
    gate_rel = 0.0 if z is None else 2 * (6 + np.abs(z)) * U
    v = x * (1.0 if last else sig)
    dv = np.abs(v) * ((0.0 if last else gate_rel) + 2 * U)
    v, dv = v.reshape(rows, groups, -1), np.broadcast_to(dv, x.shape).reshape(rows, groups, -1)
    if centre:
        m = v.mean(-1, keepdims=True)
        dv = dv + dv.mean(-1, keepdims=True) + 80 * U * np.abs(v).mean(-1, keepdims=True) + U * np.abs(m)
        v = v - m
    var = (v * v).mean(-1, keepdims=True) + eps
    r = 1 / np.sqrt(var)
    r_rel = ((np.abs(v) + dv) * dv).mean(-1, keepdims=True) / var + 90 * U
    y = (v * r).reshape(rows, ch)
    e = (r * dv * (1 + r_rel) + np.abs(v) * r * r_rel).reshape(rows, ch)
    w = np.ones(ch) if w is None else w
    b = np.zeros(ch) if b is None else b
    e = np.abs(w) * e + 4 * U * (np.abs(y * w) + np.abs(b))
    y = y * w + b
    if last and z is not None:
        e = np.abs(sig) * e + np.abs(y * sig) * gate_rel
        y = y * sig
    return y, e


def rounded(ref, err, dtype):
    """The bound after one rounding to `dtype`: half a step of the value, and the
    smallest subnormal's half where values reach there (fp16)."""
    floor = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}[dtype]
    return err + HALF_STEP[dtype] * (np.abs(ref) + err) + floor
