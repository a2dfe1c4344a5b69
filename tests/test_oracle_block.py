"""Pins of the state space block's oracle: closed forms, dense transitions, invariances, differences."""
import numpy as np
import pytest

from oracle import block as O


def draw(seed, B=2, T=9, H=4, G=2, dk=5, dv=3):
    r = np.random.default_rng(seed)
    return dict(x=r.normal(size=(B, T, H, dv)), dt=r.normal(size=(B, T, H)), b=r.normal(size=(B, T, G, dk)),
                c=r.normal(size=(B, T, G, dk)), a=-r.uniform(0.1, 2, H), d=r.normal(size=H), dt_bias=r.normal(size=H),
                s0=r.normal(size=(B, H, dk, dv)))


def test_softplus_and_silu_closed_forms():
    v = np.array([-800.0, -30.0, -1.0, 0.0, 2.0, 40.0, 800.0])
    sp = O.softplus(v)
    assert np.isfinite(sp).all() and sp[0] == 0 and sp[3] == np.log(2) and sp[-1] == 800
    np.testing.assert_allclose(sp - O.softplus(-v), v, rtol=1e-15, atol=1e-15)
    np.testing.assert_allclose(O.silu(v) - O.silu(-v) * -1, v * np.tanh(v / 2), rtol=1e-14, atol=1e-300)


def test_scan_against_pair_sums():
    """y_t = sum_{s<=t} exp(sum_{s<r<=t} dt_r A) dt_s (c_t . b_s) x_s + exp(sum_{r<=t} dt_r A) c_t S_0 + D x_t."""
    k = draw(1)
    y, sT = O.ssm(**k)
    dt = O.softplus(k["dt"] + k["dt_bias"])
    for n in range(2):
        for h in range(4):
            g = h // 2
            la = dt[n, :, h] * k["a"][h]
            for t in range(9):
                want = k["d"][h] * k["x"][n, t, h] + np.exp(la[:t + 1].sum()) * k["c"][n, t, g] @ k["s0"][n, h]
                for s in range(t + 1):
                    want = want + np.exp(la[s + 1:t + 1].sum()) * dt[n, s, h] * (k["c"][n, t, g] @ k["b"][n, s, g]) * k["x"][n, s, h]
                np.testing.assert_allclose(y[n, t, h], want, rtol=1e-11, atol=1e-12)


def test_scan_splits_and_groups():
    k = draw(2)
    y, sT = O.ssm(**k)
    cut = lambda lo, hi: {n: (v[:, lo:hi] if n in ("x", "dt", "b", "c") else v) for n, v in k.items()}
    y1, s1 = O.ssm(**cut(0, 4))
    y2, s2 = O.ssm(**{**cut(4, 9), "s0": s1})
    np.testing.assert_allclose(np.concatenate([y1, y2], 1), y, rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(s2, sT, rtol=1e-12, atol=1e-13)
    wide = {**k, "b": np.repeat(k["b"], 2, 2), "c": np.repeat(k["c"], 2, 2)}
    np.testing.assert_allclose(O.ssm(**wide)[0], y, rtol=1e-13)


def test_scan_without_decay_is_linear_attention():
    k = draw(3)
    k.update(a=np.zeros(4), d=None, dt_bias=None, s0=None, dt=np.ones((2, 9, 4)))
    y, _ = O.ssm(**k, apply_softplus=False)
    pair = np.tril(np.einsum("btgk,bsgk->bgts", k["c"], k["b"]))
    np.testing.assert_allclose(y, np.einsum("bhts,bshv->bthv", np.repeat(pair, 2, 1), k["x"]), rtol=1e-11, atol=1e-12)


def test_conv_against_numpy_convolve_and_split():
    r = np.random.default_rng(4)
    x, taps, bias, kept = r.normal(size=(2, 11, 3)), r.normal(size=(3, 4)), r.normal(size=3), r.normal(size=(2, 3, 3))
    y, last = O.short_conv(x, taps, bias, kept)
    for n in range(2):
        for ch in range(3):
            row = np.concatenate([kept[n, :, ch], x[n, :, ch]])
            u = np.convolve(row, taps[ch, ::-1], "valid") + bias[ch]
            np.testing.assert_allclose(y[n, :, ch], O.silu(u), rtol=1e-12, atol=1e-13)
    np.testing.assert_array_equal(last, x[:, -3:])
    y1, k1 = O.short_conv(x[:, :2], taps, bias, kept)
    np.testing.assert_array_equal(k1, np.concatenate([kept[:, 2:], x[:, :2]], 1))
    y2, _ = O.short_conv(x[:, 2:], taps, bias, k1)
    np.testing.assert_allclose(np.concatenate([y1, y2], 1), y, rtol=1e-13)


def test_layer_norm_properties():
    r = np.random.default_rng(5)
    x = r.normal(size=(6, 17)) + 3
    one = np.ones(17)
    y, mean, rstd = O.layer_norm(x, one, eps=0.0)
    np.testing.assert_allclose(y.mean(-1), 0, atol=1e-14)
    np.testing.assert_allclose((y * y).mean(-1), 1, rtol=1e-13)
    np.testing.assert_allclose(O.layer_norm(5 * x - 7, one, eps=0.0)[0], y, rtol=1e-12, atol=1e-13)


@pytest.mark.parametrize("width", [1, 2, 9])
def test_layer_norm_gradients_against_differences(width):
    r = np.random.default_rng(6)
    x, g, b, dy = r.normal(size=(3, width)), r.normal(size=width), r.normal(size=width), r.normal(size=(3, width))
    f = lambda x, g, b: (dy * O.layer_norm(x, g, b, 1e-3)[0]).sum()
    _, mean, rstd = O.layer_norm(x, g, b, 1e-3)
    dx, dg, db = O.layer_norm_bwd(dy, x, g, mean, rstd)
    h = 1e-6
    for got, i in ((dx, 0), (dg, 1), (db, 2)):
        args = [x, g, b]
        for at in np.ndindex(args[i].shape):
            hi, lo = [v.copy() for v in args], [v.copy() for v in args]
            hi[i][at] += h
            lo[i][at] -= h
            assert abs((f(*hi) - f(*lo)) / (2 * h) - got[at]) <= 1e-6 * max(1, abs(got).max()) * 30
