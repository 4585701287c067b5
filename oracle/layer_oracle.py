"""Float64 oracle of the layer operators (test infrastructure, plain numpy).

Rotary positions, linear attention with one decay per head (token by token)
and the norms around a block, each with its gradient written from its own
formula.  Arrays are float64; nothing here is shared with the library.
"""
from __future__ import annotations

import numpy as np


def rotary_frequencies(rot, base=10000.0, scaling="plain", factor=1.0, original=0):
    out = []
    m = 1.0
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    for i in range(rot // 2):
        f = 1.0 / base ** (2 * i / rot)
        if scaling == "linear":
            f /= factor
        if scaling == "yarn":
            turns = original * f / (2 * np.pi)
            share = min(1.0, max(0.0, (turns - 1.0) / (32.0 - 1.0)))
            f = share * f + (1.0 - share) * f / factor
            m = 0.1 * np.log(factor) + 1.0
        out.append(f)
    return np.array(out), m


def rotary(x, positions, inv_freq, m=1.0, interleaved=False, inverse=False):
    """x [B, H, T, d], positions [B, T]: each pair times a 2 x 2 rotation."""
    half = len(inv_freq)
    y = np.array(x, dtype=np.float64)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        ang = positions.astype(np.float64) * inv_freq[i]
        c, s = m * np.cos(ang)[:, None], m * np.sin(ang)[:, None]
        if inverse:
            s = -s
        xa, xb = x[..., a], x[..., b]
        y[..., a] = xa * c - xb * s
        y[..., b] = xa * s + xb * c
    return y


def linear_forward(q, k, v, loggate, S0=None, scale=1.0):
    """One sequence, token by token: q, k [Hk, n, d], v [Hv, n, dv], loggate
    [Hv], S0 [Hv, dv, d]; returns o [Hv, n, dv] and the last state."""
    Hv, n, dv = v.shape
    rep = Hv // k.shape[0]
    q, k = np.repeat(q, rep, 0), np.repeat(k, rep, 0)
    a = np.exp(loggate)[:, None, None]
    S = np.zeros((Hv, dv, k.shape[2])) if S0 is None else np.array(S0, dtype=np.float64)
    o = np.zeros((Hv, n, dv))
    for t in range(n):
        S = a * S + v[:, t, :, None] * k[:, t, None, :]
        o[:, t] = scale * np.einsum("hvk,hk->hv", S, q[:, t])
    return o, S


def linear_backward(q, k, v, loggate, S0, dO, dS, scale=1.0):
    """Gradients of sum(o dO) + sum(S_n dS): dq, dk, dv, dS0."""
    Hv, n, dv = v.shape
    Hk, _, d = k.shape
    rep = Hv // Hk
    q, k = np.repeat(q, rep, 0), np.repeat(k, rep, 0)
    a = np.exp(loggate)[:, None, None]
    S = np.zeros((Hv, dv, d)) if S0 is None else np.array(S0, dtype=np.float64)
    states = []
    for t in range(n):
        S = a * S + v[:, t, :, None] * k[:, t, None, :]
        states.append(S)
    E = np.zeros((Hv, dv, d)) if dS is None else np.array(dS, dtype=np.float64)
    dq, dk, dvv = np.zeros((Hv, n, d)), np.zeros((Hv, n, d)), np.zeros((Hv, n, dv))
    for t in reversed(range(n)):
        E = E + scale * dO[:, t, :, None] * q[:, t, None, :]
        dq[:, t] = scale * np.einsum("hvk,hv->hk", states[t], dO[:, t])
        dk[:, t] = np.einsum("hvk,hv->hk", E, v[:, t])
        dvv[:, t] = np.einsum("hvk,hk->hv", E, k[:, t])
        E = a * E
    share = lambda x: x.reshape(Hk, rep, n, d).sum(1)
    return share(dq), share(dk), dvv, E


def _act(z, act):
    s = 1.0 / (1.0 + np.exp(-z))
    return (z * s, s + z * s * (1.0 - s)) if act == "silu" else (s, s * (1.0 - s))


def block_norm(y, z, w_post, r, w_pre, scale=1.0, eps=1e-6, act="silu"):
    """y [rows, H, d], the others [rows, H d] or None: x and N (or None)."""
    rows, H, d = y.shape
    n = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) if w_post is not None else y
    n = n.reshape(rows, H * d)
    if w_post is not None:
        n = n * w_post
    x = scale * (n if z is None else n * _act(z, act)[0])
    if r is not None:
        x = x + r
    if w_pre is None:
        return x, None
    return x, w_pre * x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)


def block_norm_backward(y, z, w_post, r, w_pre, dX, dN, scale=1.0, eps=1e-6, act="silu"):
    """dy [rows, H, d], dz, dr [rows, H d], dw_post, dw_pre (None where absent)."""
    rows, H, d = y.shape
    W = H * d
    x, _ = block_norm(y, z, w_post, r, w_pre, scale, eps, act)
    dx = np.zeros((rows, W)) if dX is None else np.array(dX)
    dw_pre = dw_post = dz = None
    if w_pre is not None:
        v = (x * x).mean(-1, keepdims=True) + eps
        dw_pre = (dN * x / np.sqrt(v)).sum(0)
        g = dN * w_pre
        dx = dx + g / np.sqrt(v) - x * (g * x).sum(-1, keepdims=True) / (W * v ** 1.5)
    dr = dx if r is not None else None
    dn = scale * dx
    v = (y * y).mean(-1, keepdims=True) + eps
    yh = (y / np.sqrt(v) if w_post is not None else y).reshape(rows, W)
    n = yh * w_post if w_post is not None else yh
    if z is not None:
        g, slope = _act(z, act)
        dz = dn * n * slope
        dn = dn * g
    if w_post is None:
        return dn.reshape(rows, H, d), dz, dr, None, dw_pre
    dw_post = (dn * yh).sum(0)
    e = (dn * w_post).reshape(rows, H, d)
    dy = e / np.sqrt(v) - y * (e * y).sum(-1, keepdims=True) / (d * v ** 1.5)
    return dy, dz, dr, dw_post, dw_pre
