"""float64 oracles of the operators around the scans, from their definitions, token by token.

The norm of queries and keys with rotary positions, the gated linear recurrence and the gated
feed-forward block, each with its gradients derived by hand (the tests check them against
differences). NumPy only; shares nothing with the GPU path.
"""

from __future__ import annotations

import math

import numpy as np


def _f64(x):
    return None if x is None else np.asarray(x, np.float64)


# ---- queries and keys ---------------------------------------------------------------------


def _pairs(rot, layout):
    i = np.arange(rot // 2)
    return (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)


def _norm(x, norm, eps):
    if norm == "rms":
        return np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    if norm == "l2":
        return np.sqrt(np.sum(x * x, -1, keepdims=True) + eps)
    return np.ones_like(x[..., :1])


def norm_rope(x, positions, freqs, magnitude=1.0, norm="rms", eps=1e-6, layout="half", weight=None):
    """Rows x [batch, heads, tokens, width], positions [batch, tokens]."""
    x, freqs = _f64(x), _f64(freqs)
    y = x / _norm(x, norm, eps)
    if weight is not None:
        y = y * _f64(weight)
    if freqs is None or len(freqs) == 0:
        return y
    a, b = _pairs(2 * len(freqs), layout)
    angle = np.asarray(positions, np.float64)[:, None, :, None] * freqs
    c, s = magnitude * np.cos(angle), magnitude * np.sin(angle)
    out = y.copy()
    out[..., a] = y[..., a] * c - y[..., b] * s
    out[..., b] = y[..., b] * c + y[..., a] * s
    return out


def norm_rope_backward(dy, x, positions, freqs, magnitude=1.0, norm="rms", eps=1e-6, layout="half", weight=None):
    """(dx, dweight); dweight is None without a weight."""
    dy, x, freqs = _f64(dy), _f64(x), _f64(freqs)
    e = dy.copy()
    if freqs is not None and len(freqs):
        a, b = _pairs(2 * len(freqs), layout)
        angle = np.asarray(positions, np.float64)[:, None, :, None] * freqs
        c, s = magnitude * np.cos(angle), magnitude * np.sin(angle)
        e[..., a] = dy[..., a] * c + dy[..., b] * s
        e[..., b] = dy[..., b] * c - dy[..., a] * s
    size = _norm(x, norm, eps)
    dw = None
    if weight is not None:
        dw = np.sum(e * x / size, axis=(0, 1, 2))
        e = e * _f64(weight)
    if norm == "none":
        return e, dw
    n = x.shape[-1] if norm == "rms" else 1
    return e / size - x * np.sum(e * x, -1, keepdims=True) / (n * size ** 3), dw


# ---- the gated recurrence -------------------------------------------------------------------


def gated_scan(q, k, v, g, scale=1.0, S0=None):
    """(o, S after the last token, S before every token [batch, heads, tokens, 64, 64])."""
    q, k, v, g = _f64(q), _f64(k), _f64(v), _f64(g)
    B, H, T, D = q.shape
    S = np.zeros((B, H, D, D)) if S0 is None else _f64(S0).copy()
    o, before = np.zeros(q.shape), np.zeros((B, H, T, D, D))
    for t in range(T):
        before[:, :, t] = S
        S = np.exp(g[:, :, t])[..., None, None] * S + k[:, :, t, :, None] * v[:, :, t, None, :]
        o[:, :, t] = scale * np.einsum("bha,bhac->bhc", q[:, :, t], S)
    return o, S, before


def gated_scan_backward(do, q, k, v, g, scale=1.0, S0=None, dS=None):
    """(dq, dk, dv, dg, dS0)."""
    do, q, k, v, g = _f64(do), _f64(q), _f64(k), _f64(v), _f64(g)
    _, S, before = gated_scan(q, k, v, g, scale, S0)
    B, H, T, D = q.shape
    dS = np.zeros((B, H, D, D)) if dS is None else _f64(dS).copy()
    dq, dk, dv, dg = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape), np.zeros(g.shape)
    for t in range(T - 1, -1, -1):
        after = S if t == T - 1 else before[:, :, t + 1]
        dq[:, :, t] = scale * np.einsum("bhac,bhc->bha", after, do[:, :, t])
        dS = dS + scale * q[:, :, t, :, None] * do[:, :, t, None, :]
        dk[:, :, t] = np.einsum("bhac,bhc->bha", dS, v[:, :, t])
        dv[:, :, t] = np.einsum("bhac,bha->bhc", dS, k[:, :, t])
        f = np.exp(g[:, :, t])
        dg[:, :, t] = f * np.sum(dS * before[:, :, t], axis=(-1, -2))
        dS = f[..., None, None] * dS
    return dq, dk, dv, dg, dS


# ---- the gated feed-forward block -------------------------------------------------------------

_erf = np.vectorize(math.erf, otypes=[np.float64])


def activation(x, kind):
    """(act(x), act'(x))."""
    if kind == "silu":
        s = 1.0 / (1.0 + np.exp(-x))
        return x * s, s * (1.0 + x * (1.0 - s))
    phi = 0.5 * (1.0 + _erf(x / math.sqrt(2.0)))
    return x * phi, phi + x * np.exp(-0.5 * x * x) / math.sqrt(2.0 * math.pi)


def gated_ffn(x, wg, wu, kind="silu"):
    """(z, gate, up)."""
    x, wg, wu = _f64(x), _f64(wg), _f64(wu)
    g, u = x @ wg.T, x @ wu.T
    return activation(g, kind)[0] * u, g, u


def gated_ffn_backward(dz, x, wg, wu, g, u, kind="silu"):
    """(dx, dwg, dwu, dg, du) from the given pre-activations."""
    dz, x, wg, wu, g, u = (_f64(t) for t in (dz, x, wg, wu, g, u))
    a, da = activation(g, kind)
    dg, du = dz * u * da, dz * a
    return dg @ wg + du @ wu, dg.T @ x, du.T @ x, dg, du
