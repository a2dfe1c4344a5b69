"""Pins of the attention block's oracle, each against something that does not share its formulas."""
import math

import numpy as np
import pytest

from oracle import attention as A


def rng(seed):
    return np.random.default_rng(seed)


def brute(q, k, v, window, scale):
    """Pair by pair, with Python numbers."""
    T, H, d = q.shape
    S, G = k.shape[:2]
    o, lse = np.zeros((T, H, d)), np.full((T, H), -math.inf)
    for t in range(T):
        for h in range(H):
            g = h // (H // G)
            seen = [j for j in range(S) if j <= S - T + t and (window is None or j > S - T + t - window)]
            w = [math.exp(scale * sum(float(a) * float(b) for a, b in zip(q[t, h], k[j, g]))) for j in seen]
            if w:
                lse[t, h] = math.log(sum(w))
                for c in range(d):
                    o[t, h, c] = sum(x * float(v[j, g, c]) for x, j in zip(w, seen)) / sum(w)
    return o, lse


@pytest.mark.parametrize("T,S,H,G,window", [(1, 1, 1, 1, None), (3, 7, 2, 1, None), (5, 5, 4, 2, 2), (6, 3, 2, 2, None), (4, 9, 3, 1, 1)])
def test_attention_pair_by_pair(T, S, H, G, window):
    r = rng(T * 10 + S)
    q, k, v = r.normal(size=(T, H, 4)), r.normal(size=(S, G, 4)), r.normal(size=(S, G, 4))
    o, lse = A.attention(q, k, v, window, 0.7)
    ob, lb = brute(q, k, v, window, 0.7)
    np.testing.assert_allclose(o, ob, rtol=1e-12, atol=1e-14)
    np.testing.assert_allclose(lse, lb, rtol=1e-12)


def test_attention_closed_forms():
    r = rng(3)
    k, v = r.normal(size=(6, 1, 8)), r.normal(size=(6, 1, 8))
    o, lse = A.attention(np.zeros((6, 2, 8)), k, v)  # equal scores: running means
    means = np.cumsum(v[:, 0], 0) / np.arange(1, 7)[:, None]
    np.testing.assert_allclose(o[:, 0], means, rtol=1e-13)
    np.testing.assert_allclose(lse[:, 1], np.log(np.arange(1, 7)), atol=1e-14)
    o, _ = A.attention(r.normal(size=(6, 2, 8)), k, v, window=1)  # a window of one: the value itself
    np.testing.assert_allclose(o[:, 1], v[:, 0], rtol=1e-13)


def test_attention_gradients_against_differences():
    r = rng(5)
    T, S, H, G, d, window = 5, 7, 4, 2, 3, 4
    q, k, v, w = r.normal(size=(T, H, d)), r.normal(size=(S, G, d)), r.normal(size=(S, G, d)), r.normal(size=(T, H, d))
    o, lse = A.attention(q, k, v, window)
    grads = A.attention_bwd(w, q, k, v, o, lse, window)
    for x, g in zip((q, k, v), grads):
        for at in [tuple(r.integers(0, n) for n in x.shape) for _ in range(12)]:
            old = x[at]
            x[at] = old + 1e-5
            up = (w * A.attention(q, k, v, window)[0]).sum()
            x[at] = old - 1e-5
            down = (w * A.attention(q, k, v, window)[0]).sum()
            x[at] = old
            assert abs((up - down) / 2e-5 - g[at]) < 1e-8, at


def test_attention_gradients_of_hidden_tokens_are_zero():
    r = rng(6)
    q, k, v, w = r.normal(size=(6, 1, 4)), r.normal(size=(3, 1, 4)), r.normal(size=(3, 1, 4)), r.normal(size=(6, 1, 4))
    o, lse = A.attention(q, k, v)
    assert np.isneginf(lse[:3]).all() and not o[:3].any()
    dq, dk, dv = A.attention_bwd(w, q, k, v, o, lse)
    assert not dq[:3].any() and np.isfinite(dk).all() and dv.any()


def test_steps_equal_a_prompt():
    r = rng(7)
    T, C, H, G, d = 23, 8, 4, 2, 4
    q, k, v = r.normal(size=(T, H, d)), r.normal(size=(T, G, d)), r.normal(size=(T, G, d))
    for window in (None, 3):
        want, _ = A.attention(q, k, v, min(C, window or C))
        kc, vc = np.full((C, G, d), 9.0), np.full((C, G, d), 9.0)
        for p in range(T):
            o, kc, vc = A.step(q[p], k[p], v[p], kc, vc, p, window)
            np.testing.assert_allclose(o, want[p], rtol=1e-12, atol=1e-14)
    o, kc2, _ = A.step(q[0], k[0], v[0], kc, vc, -1)
    assert not o.any() and (kc2 == kc).all()


def test_rotary_properties():
    r = rng(8)
    x, freq, pos = r.normal(size=(5, 2, 10)), 10.0 ** -np.arange(4), np.array([0, 1, 7, 1000, 12345])
    for inter in (False, True):
        y = A.rotary(x, freq, pos, inter)
        np.testing.assert_allclose((y ** 2).sum(-1), (x ** 2).sum(-1), rtol=1e-12)  # lengths stay
        np.testing.assert_array_equal(y[..., 8:], x[..., 8:])
        np.testing.assert_array_equal(y[0], x[0])  # position 0
        np.testing.assert_allclose(A.rotary(y, freq, pos, inter, inverse=True), x, rtol=1e-9, atol=1e-12)
        # products of a query and a key depend on the distance alone
        a, b = A.rotary(x[:1], freq, [40], inter), A.rotary(x[1:2], freq, [33], inter)
        c, d = A.rotary(x[:1], freq, [7], inter), A.rotary(x[1:2], freq, [0], inter)
        np.testing.assert_allclose((a * b).sum(), (c * d).sum(), rtol=1e-10)
    # a pair as a complex number
    y = A.rotary(x, freq, pos, True, scale=2.0)
    z = (x[..., 0:8:2] + 1j * x[..., 1:8:2]) * 2.0 * np.exp(1j * pos[:, None, None] * freq)
    np.testing.assert_allclose(y[..., 0:8:2] + 1j * y[..., 1:8:2], z, rtol=1e-12, atol=1e-14)


def test_rms_norm_properties():
    r = rng(9)
    x, res, gamma = r.normal(size=(4, 6)), r.normal(size=(4, 6)), r.normal(size=6)
    y, h, rstd = A.rms_norm(x, np.ones(6), 0.0, res)
    np.testing.assert_allclose((y ** 2).mean(-1), 1.0, rtol=1e-13)
    np.testing.assert_allclose(A.rms_norm(5 * x, gamma, 0.0, 5 * res)[0], A.rms_norm(x, gamma, 0.0, res)[0], rtol=1e-12)
    assert A.rms_norm(np.zeros((1, 4)), np.ones(4), 1e-6)[2] == pytest.approx(1e3)
    w, dh, eps = r.normal(size=(4, 6)), r.normal(size=(4, 6)), 0.3
    _, h, rstd = A.rms_norm(x, gamma, eps, res)
    dx, dgamma = A.rms_norm_bwd(w, h, gamma, rstd, dh)

    def loss():
        y, h, _ = A.rms_norm(x, gamma, eps, res)
        return (w * y).sum() + (dh * h).sum()

    for t, g in ((x, dx), (res, dx), (gamma, dgamma)):
        for at in [tuple(r.integers(0, n) for n in t.shape) for _ in range(6)]:
            old = t[at]
            t[at] = old + 1e-5
            up = loss()
            t[at] = old - 1e-5
            down = loss()
            t[at] = old
            assert abs((up - down) / 2e-5 - g[at]) < 1e-8
