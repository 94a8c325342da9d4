"""Pins of the layer operators' FP64 oracle (CPU): central differences of
<dy, y> + <dfinal, final> for every input, closed forms, and split calls.

Tolerance of the differences: step 1e-5 in 64 bits leaves a truncation of about
1e-10 and a rounding of about 1e-16 / 1e-5 = 1e-11 relative to values of order
one: 1e-6 of the gradient's size.
"""

import numpy as np
import pytest

from oracle import layer

EPS = 1e-5


def numeric(f, v):
    g = np.zeros_like(v)
    it = np.nditer(v, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        old = v[i]
        v[i] = old + EPS
        hi = f()
        v[i] = old - EPS
        lo = f()
        v[i] = old
        g[i] = (hi - lo) / (2 * EPS)
    return g


def close(a, b):
    assert np.max(np.abs(a - b)) <= 1e-6 * max(1.0, np.max(np.abs(b)))


@pytest.mark.parametrize("W,silu,starts", [(4, True, [0, 2, 2, 9]), (3, False, [0, 1, 6]), (2, True, [0, 5])])
def test_conv_gradients(W, silu, starts):
    rng = np.random.default_rng(1)
    T, D, N = starts[-1], 3, len(starts) - 1
    x, w, bias = rng.normal(size=(T, D)), rng.normal(size=(D, W)), rng.normal(size=D)
    h0, dy, df = rng.normal(size=(N, W - 1, D)), rng.normal(size=(T, D)), rng.normal(size=(N, W - 1, D))
    r = layer.conv(x, w, bias, h0, starts, silu, dy, df)

    def loss():
        o = layer.conv(x, w, bias, h0, starts, silu)
        return np.sum(o["y"] * dy) + np.sum(o["final"] * df)

    for name, v in (("dx", x), ("dweight", w), ("dbias", bias), ("dinit", h0)):
        close(r[name], numeric(loss, v))


def test_conv_of_one_tap_history():
    x = np.arange(1.0, 5.0)[:, None]
    o = layer.conv(x, np.array([[10.0, 1.0]]), None, None, [0, 1, 4], False)
    assert o["y"][:, 0].tolist() == [1.0, 2.0, 23.0, 34.0]
    assert o["final"][:, 0, 0].tolist() == [1.0, 4.0]


@pytest.mark.parametrize("G,gate,sp,starts", [(1, True, True, [0, 3, 3, 7]), (2, False, False, [0, 4])])
def test_scan_gradients(G, gate, sp, starts):
    rng = np.random.default_rng(2)
    T, D, S, N = starts[-1], 4, 3, len(starts) - 1
    x, dt = rng.normal(size=(T, D)), rng.normal(size=(T, D)) * 0.3 + (0.0 if sp else 0.6)
    A, b, c = rng.normal(size=(D, S)) * 0.4, rng.normal(size=(T, G, S)), rng.normal(size=(T, G, S))
    skip, bias, h0 = rng.normal(size=D), rng.normal(size=D) * 0.2, rng.normal(size=(N, D, S))
    z = rng.normal(size=(T, D)) if gate else None
    dy, dht = rng.normal(size=(T, D)), rng.normal(size=(N, D, S))
    r = layer.scan(x, dt, A, b, c, skip, z, bias, h0, starts, sp, dy, dht)

    def loss():
        o = layer.scan(x, dt, A, b, c, skip, z, bias, h0, starts, sp)
        return np.sum(o["y"] * dy) + np.sum(o["ht"] * dht)

    pairs = [("dx", x), ("ddt", dt), ("dA_log", A), ("db", b), ("dc", c), ("dd_skip", skip), ("ddt_bias", bias),
             ("dh0", h0)] + ([("dz", z)] if gate else [])
    for name, v in pairs:
        close(r[name], numeric(loss, v))


def test_scan_single_token_and_split_calls():
    rng = np.random.default_rng(3)
    T, D, S = 9, 2, 3
    x, dt, A = rng.normal(size=(T, D)), rng.normal(size=(T, D)), rng.normal(size=(D, S))
    b, c, h0 = rng.normal(size=(T, 1, S)), rng.normal(size=(T, 1, S)), rng.normal(size=(1, D, S))
    one = layer.scan(x[:1], dt[:1], A, b[:1], c[:1], None, None, None, h0, [0, 1])
    dl = np.log1p(np.exp(dt[0]))
    h = np.exp(-dl[:, None] * np.exp(A)) * h0[0] + (dl * x[0])[:, None] * b[0]
    assert np.allclose(one["ht"][0], h, rtol=1e-13) and np.allclose(one["y"][0], h @ c[0, 0], rtol=1e-12)
    whole = layer.scan(x, dt, A, b, c, None, None, None, h0, [0, T])
    p = layer.scan(x[:4], dt[:4], A, b[:4], c[:4], None, None, None, h0, [0, 4])
    q = layer.scan(x[4:], dt[4:], A, b[4:], c[4:], None, None, None, p["ht"], [0, T - 4])
    assert np.allclose(np.concatenate([p["y"], q["y"]]), whole["y"]) and np.allclose(q["ht"], whole["ht"])


def test_norm_gradients():
    rng = np.random.default_rng(4)
    x, w, dy, dres = rng.normal(size=(3, 7)), rng.normal(size=7), rng.normal(size=(3, 7)), rng.normal(size=(3, 7))
    r = layer.norm(x, w, None, 1e-3, dy, dres)

    def loss():
        return np.sum(layer.norm(x, w, None, 1e-3)["y"] * dy) + np.sum(x * dres)

    close(r["dx"], numeric(loss, x))
    close(r["dweight"], numeric(loss, w))
    assert np.allclose(np.mean(layer.norm(x, np.ones(7), None, 0.0)["y"] ** 2, axis=1), 1.0)
