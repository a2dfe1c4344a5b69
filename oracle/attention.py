"""fp64 CPU oracle of the attention block -- TEST INFRASTRUCTURE.

Plain numpy in float64, the definitions written out: causal attention with shared key heads and a
window, its gradients, one token over a cache, rotary positions, and the root-mean-square norm with
its gradients.  It shares no code with the HIP library and never imports it.

Parity status: pinned by tests/test_oracle_attention.py (closed forms, brute force over pairs,
invariances and central differences).
"""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0


def _f64(x):
    if x is None:
        return None
    if hasattr(x, "detach"):
        x = x.detach().cpu().double().numpy()
    return np.asarray(x, dtype=np.float64)


def sees(T, S, window=None):
    """[T,S]: query t stands at S - T + t and sees the keys at and before it, the last `window` of them."""
    ago = (S - T + np.arange(T))[:, None] - np.arange(S)[None, :]
    return (ago >= 0) & (ago < (window or S + T + 1))


def scores(q, k, window=None, scale=None):
    """One sequence: q [T,H,d], k [S,G,d] -> [H,T,S], minus infinity where a query does not see."""
    q, k = _f64(q), _f64(k)
    T, H, d = q.shape
    S, G = k.shape[:2]
    kk = np.repeat(k, H // G, axis=1)
    s = np.einsum("thd,shd->hts", q, kk) * (d ** -0.5 if scale is None else scale)
    return np.where(sees(T, S, window)[None], s, -np.inf)


def attention(q, k, v, window=None, scale=None):
    """One sequence: o [T,H,d], lse [T,H].  A query that sees nothing has o = 0 and lse = -inf."""
    v = _f64(v)
    s = scores(q, k, window, scale)
    H, G = s.shape[0], v.shape[1]
    with np.errstate(divide="ignore"):
        m = s.max(-1, initial=-np.inf)
        ref = np.where(np.isfinite(m), m, 0.0)
        p = np.exp(s - ref[..., None])
        l = p.sum(-1)
        lse = np.where(l > 0, ref + np.log(l), -np.inf)
    o = np.einsum("hts,shd->thd", p / np.where(l > 0, l, 1.0)[..., None], np.repeat(v, H // G, axis=1))
    return o, lse.T


def attention_bwd(d_o, q, k, v, o, lse, window=None, scale=None):
    """One sequence: dq, dk, dv of sum(d_o * o), from o and lse as they are given."""
    d_o, q, k, v, o, lse = (_f64(x) for x in (d_o, q, k, v, o, lse))
    T, H, d = q.shape
    S, G = k.shape[:2]
    scale = d ** -0.5 if scale is None else scale
    kk, vv = np.repeat(k, H // G, axis=1), np.repeat(v, H // G, axis=1)
    seen = sees(T, S, window)[None]
    s = np.einsum("thd,shd->hts", q, kk) * scale
    p = np.where(seen, np.exp(np.where(seen, s - np.where(np.isfinite(lse), lse, 0.0).T[..., None], 0.0)), 0.0)
    dp = np.einsum("thd,shd->hts", d_o, vv)
    ds = p * (dp - (d_o * o).sum(-1).T[..., None])
    dq = np.einsum("hts,shd->thd", ds, kk) * scale
    dk = (np.einsum("hts,thd->shd", ds, q) * scale).reshape(S, G, H // G, d).sum(2)
    dv = np.einsum("hts,thd->shd", p, d_o).reshape(S, G, H // G, d).sum(2)
    return dq, dk, dv


def step(q, k, v, k_cache, v_cache, pos, window=None, scale=None):
    """One token of one sequence: q [H,d], k, v [G,d], caches [C,G,d]; returns o and the two caches."""
    q, k, v, kc, vc = (_f64(x) for x in (q, k, v, k_cache, v_cache))
    kc, vc = kc.copy(), vc.copy()
    if pos < 0:
        return np.zeros(q.shape), kc, vc
    C = kc.shape[0]
    kc[pos % C], vc[pos % C] = k, v
    tokens = np.arange(max(0, pos + 1 - min(C, window or C)), pos + 1) % C
    o, _ = attention(q[None], kc[tokens], vc[tokens], None, scale)
    return o[0], kc, vc


def rotary(x, freq, positions, interleaved=False, inverse=False, scale=1.0):
    """x [...,heads,d], positions [...]: the first 2 len(freq) channels turned."""
    x, freq = _f64(x), _f64(freq)
    n = freq.shape[0]
    t = np.asarray(positions, dtype=np.float64)[..., None, None] * freq
    c, s = np.cos(t) * scale, np.sin(t) * (-scale if inverse else scale)
    y = x.copy()
    a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def rms_norm(x, gamma, eps, residual=None):
    """y, h, rstd over the last axis."""
    h = _f64(x) if residual is None else _f64(x) + _f64(residual)
    rstd = 1.0 / np.sqrt((h * h).mean(-1) + eps)
    return h * rstd[..., None] * _f64(gamma), h, rstd


def rms_norm_bwd(dy, h, gamma, rstd, dh=None):
    """dx, dgamma of sum(dy * y) + sum(dh * h), from rstd as it is given."""
    dy, h, gamma, rstd = (_f64(t) for t in (dy, h, gamma, rstd))
    u, v = h * rstd[..., None], dy * gamma
    dx = rstd[..., None] * (v - u * (u * v).mean(-1, keepdims=True))
    if dh is not None:
        dx = dx + _f64(dh)
    return dx, (dy * u).reshape(-1, h.shape[-1]).sum(0)
