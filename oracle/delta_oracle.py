"""Float64 definitions of the gated delta rule and of the query/key norm and
rotation, step by step in NumPy, with the gradients written out from the
formulas. Shares no code with the kernels.

Layouts: q, k [B, L, Hk, Dk], v [B, L, Hv, Dv], g, beta [B, L, Hv], states
[B, Hv, Dk, Dv]; value head h reads query/key head h // (Hv // Hk).
"""

from __future__ import annotations

import math

import numpy as np


def _prepare(q, k, v, g, beta, s0, lengths):
    q, k, v, g, beta = (np.asarray(x, dtype=np.float64) for x in (q, k, v, g, beta))
    B, L, Hv, Dv = v.shape
    n = Hv // k.shape[2]
    live = np.arange(L)[None, :] < (np.full(B, L) if lengths is None else np.clip(lengths, 0, L))[:, None]
    m4 = live[:, :, None, None]
    q, k = (np.where(m4, np.repeat(x, n, axis=2), 0.0) for x in (q, k))
    v = np.where(m4, v, 0.0)
    a = np.where(live[:, :, None], np.exp(g), 1.0)
    beta = np.where(live[:, :, None], beta, 0.0)
    S = np.zeros((B, Hv, k.shape[3], Dv)) if s0 is None else np.array(s0, dtype=np.float64)
    return q, k, v, a, beta, S, live, n


def gated_delta(q, k, v, g, beta, s0=None, scale=None, lengths=None):
    """(y, s_last); rows of y behind a sequence's length are zero."""
    scale = np.shape(k)[-1] ** -0.5 if scale is None else scale
    q, k, v, a, beta, S, live, _ = _prepare(q, k, v, g, beta, s0, lengths)
    y = np.zeros_like(v)
    for t in range(v.shape[1]):
        S = a[:, t, :, None, None] * S
        u = beta[:, t, :, None] * (v[:, t] - np.einsum("bhkv,bhk->bhv", S, k[:, t]))
        S = S + k[:, t, :, :, None] * u[:, :, None, :]
        y[:, t] = scale * np.einsum("bhkv,bhk->bhv", S, q[:, t])
    return np.where(live[:, :, None, None], y, 0.0), S


def gated_delta_backward(dy, q, k, v, g, beta, s0=None, ds_last=None, scale=None, lengths=None):
    """(dq, dk, dv, dg, dbeta, ds0); rows behind a length are zero."""
    scale = np.shape(k)[-1] ** -0.5 if scale is None else scale
    q, k, v, a, beta, S, live, n = _prepare(q, k, v, g, beta, s0, lengths)
    B, L, Hv, Dv = v.shape
    dy = np.where(live[:, :, None, None], np.asarray(dy, dtype=np.float64), 0.0)
    decayed = []                                   # a_t S_{t-1}
    for t in range(L):
        S = a[:, t, :, None, None] * S
        decayed.append(S)
        u = beta[:, t, :, None] * (v[:, t] - np.einsum("bhkv,bhk->bhv", S, k[:, t]))
        S = S + k[:, t, :, :, None] * u[:, :, None, :]
    D = np.zeros_like(S) if ds_last is None else np.array(ds_last, dtype=np.float64)
    dq, dk, dv, dg, db = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v), np.zeros_like(beta), np.zeros_like(beta)
    for t in range(L - 1, -1, -1):
        Sd = decayed[t]
        e = v[:, t] - np.einsum("bhkv,bhk->bhv", Sd, k[:, t])
        u = beta[:, t, :, None] * e
        St = Sd + k[:, t, :, :, None] * u[:, :, None, :]
        o = scale * dy[:, t]
        dq[:, t] = np.einsum("bhkv,bhv->bhk", St, o)
        D = D + q[:, t, :, :, None] * o[:, :, None, :]
        du = np.einsum("bhkv,bhk->bhv", D, k[:, t])
        db[:, t] = np.einsum("bhv,bhv->bh", du, e)
        de = beta[:, t, :, None] * du
        dv[:, t] = de
        dk[:, t] = np.einsum("bhkv,bhv->bhk", D, u) - np.einsum("bhkv,bhv->bhk", Sd, de)
        D = D - k[:, t, :, :, None] * de[:, :, None, :]
        dg[:, t] = np.einsum("bhkv,bhkv->bh", D, Sd)
        D = a[:, t, :, None, None] * D
    dq, dk = (x.reshape(B, L, Hv // n, n, -1).sum(axis=3) for x in (dq, dk))
    m3 = live[:, :, None]
    return (np.where(m3[..., None], dq, 0.0), np.where(m3[..., None], dk, 0.0), np.where(m3[..., None], dv, 0.0),
            np.where(m3, dg, 0.0), np.where(m3, db, 0.0), D)


def _rotation(D, freqs, positions, rope_scale, interleaved):
    """The rotation of each token as a matrix [..., D, D]: y = M x."""
    R = 0 if freqs is None else 2 * len(freqs)
    pos = np.asarray(positions, dtype=np.float64)
    M = np.zeros(pos.shape + (D, D))
    for j in range(R // 2):
        e, f = (2 * j, 2 * j + 1) if interleaved else (j, j + R // 2)
        c, s = rope_scale * np.cos(pos * freqs[j]), rope_scale * np.sin(pos * freqs[j])
        M[..., e, e], M[..., e, f], M[..., f, e], M[..., f, f] = c, -s, s, c
    for j in range(R, D):
        M[..., j, j] = 1.0
    return M


def _default_positions(x, positions):
    lead = x.shape[:-2]
    return np.broadcast_to(np.arange(lead[-1]), lead) if positions is None else positions


def norm_rope(x, norm, weight=None, eps=1e-6, freqs=None, positions=None, rope_scale=1.0, interleaved=False):
    """One of q and k: x [..., heads, D], positions [...] or None."""
    x = np.asarray(x, dtype=np.float64)
    if norm is not None:
        m = (x ** 2).sum(-1, keepdims=True) / (x.shape[-1] if norm == "rms" else 1)
        x = x / np.sqrt(m + eps)
    if weight is not None:
        x = x * np.asarray(weight, dtype=np.float64)
    M = _rotation(x.shape[-1], freqs, _default_positions(x, positions), rope_scale, interleaved)
    return np.einsum("...ij,...hj->...hi", M, x)


def norm_rope_backward(dy, x, norm, weight=None, eps=1e-6, freqs=None, positions=None, rope_scale=1.0,
                       interleaved=False):
    """(dx, dweight), dweight None without a weight."""
    x, d = np.asarray(x, dtype=np.float64), np.asarray(dy, dtype=np.float64)
    D = x.shape[-1]
    M = _rotation(D, freqs, _default_positions(x, positions), rope_scale, interleaved)
    d = np.einsum("...ij,...hi->...hj", M, d)
    if norm is None:
        return d, None
    n = D if norm == "rms" else 1
    root = np.sqrt((x ** 2).sum(-1, keepdims=True) / n + eps)
    dw = None
    if weight is not None:
        dw = (d * x / root).reshape(-1, D).sum(0)
        d = d * np.asarray(weight, dtype=np.float64)
    return d / root - x * (d * x).sum(-1, keepdims=True) / (n * root ** 3), dw


def rope_frequency(j, R, base, factor=1.0, scaling=None, original_length=None, fast=32.0, slow=1.0):
    """Radians per position of pair j."""
    if scaling == "base":
        base = base * factor ** (R / (R - 2))
    f = base ** (-2.0 * j / R)
    if scaling == "linear":
        return f / factor
    if scaling == "parts":
        turns = original_length * f / (2 * math.pi)
        if turns >= fast:
            return f
        if turns <= slow:
            return f / factor
        keep = (turns - slow) / (fast - slow)
        return keep * f + (1 - keep) * f / factor
    return f
