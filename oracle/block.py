"""fp64 CPU oracle of the state space block -- TEST INFRASTRUCTURE.

Plain numpy in float64, the definitions written out: the selective state space scan token by
token, the causal convolution tap by tap, layer norm and its gradients.  It shares no code with
the HIP library and never imports it.

Parity status: pinned by tests/test_oracle_block.py (closed forms, dense transition products,
numpy.convolve, invariances and central differences).
"""
from __future__ import annotations

import numpy as np

TAPS = 4


def _f64(x):
    if x is None:
        return None
    if hasattr(x, "detach"):
        x = x.detach().cpu().double().numpy()
    return np.asarray(x, dtype=np.float64)


def softplus(v):
    v = _f64(v)
    return np.maximum(v, 0.0) + np.log1p(np.exp(-np.abs(v)))


def silu(v):
    v = _f64(v)
    e = np.exp(-np.abs(v))
    return v * np.where(v >= 0, 1.0, e) / (1.0 + e)


def ssm(x, dt, b, c, a, d=None, dt_bias=None, s0=None, apply_softplus=True):
    """x [B,T,H,dv], dt [B,T,H], b, c [B,T,G,dk], a, d, dt_bias [H], s0 [B,H,dk,dv].
    Returns y [B,T,H,dv] and the final state."""
    x, dt, b, c, a, d, dt_bias, s0 = (_f64(v) for v in (x, dt, b, c, a, d, dt_bias, s0))
    B, T, H, dv = x.shape
    G, dk = b.shape[2:]
    step = dt if dt_bias is None else dt + dt_bias
    if apply_softplus:
        step = softplus(step)
    group = np.arange(H) // (H // G)
    s = np.zeros((B, H, dk, dv)) if s0 is None else s0.copy()
    y = np.empty((B, T, H, dv))
    for t in range(T):
        s = s * np.exp(step[:, t] * a)[..., None, None]
        s = s + step[:, t, :, None, None] * b[:, t, group, :, None] * x[:, t, :, None, :]
        y[:, t] = (s * c[:, t, group, :, None]).sum(-2)
    if d is not None:
        y = y + d[:, None] * x
    return y, s


def short_conv(x, taps, bias=None, kept=None):
    """x [B,T,C], taps [C,4], bias [C], kept [B,3,C].  Returns y and the last three inputs."""
    x, taps, bias, kept = (_f64(v) for v in (x, taps, bias, kept))
    B, T, C = x.shape
    row = np.concatenate([np.zeros((B, TAPS - 1, C)) if kept is None else kept, x], 1)
    u = np.zeros((B, T, C)) if bias is None else np.broadcast_to(bias, (B, T, C)).copy()
    for t in range(T):
        for j in range(TAPS):
            u[:, t] += taps[:, j] * row[:, t + j]
    return silu(u), row[:, T:T + TAPS - 1]


def layer_norm(x, gamma, beta=None, eps=1e-5):
    """x [rows,width].  Returns y, mean, rstd."""
    x, gamma, beta = (_f64(v) for v in (x, gamma, beta))
    mean = x.mean(-1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(-1) + eps)
    y = (x - mean[:, None]) * rstd[:, None] * gamma
    return (y if beta is None else y + beta), mean, rstd


def layer_norm_bwd(dy, x, gamma, mean, rstd):
    """Gradients of sum(dy * y): dx, dgamma, dbeta, from the statistics given."""
    dy, x, gamma, mean, rstd = (_f64(v) for v in (dy, x, gamma, mean, rstd))
    u = (x - mean[:, None]) * rstd[:, None]
    v = dy * gamma
    dx = rstd[:, None] * (v - v.mean(-1, keepdims=True) - u * (u * v).mean(-1, keepdims=True))
    return dx, (dy * u).sum(0), dy.sum(0)
