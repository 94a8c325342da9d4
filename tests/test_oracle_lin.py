"""Pins of the FP64 oracle of linear attention, of the rounding to 8 bits and of its
product (CPU): central differences, closed forms, and the format's own table."""

import numpy as np
import pytest
import torch

from oracle import layer
from tests.test_oracle_layer import close, numeric


@pytest.mark.parametrize("HV,decay,starts", [(2, [-0.3, 0.0], [0, 3, 3, 7]), (4, [-1.0, -0.1, 0.05, -2.0], [0, 5]),
                                             (2, None, [0, 1, 4])])
def test_lin_gradients(HV, decay, starts):
    rng = np.random.default_rng(1)
    T, H, K, V, N = starts[-1], 2, 3, 2, len(starts) - 1
    q, k, v = rng.normal(size=(T, H, K)), rng.normal(size=(T, H, K)), rng.normal(size=(T, HV, V))
    h0, do, dht = rng.normal(size=(N, HV, K, V)), rng.normal(size=(T, HV, V)), rng.normal(size=(N, HV, K, V))
    d = None if decay is None else np.array(decay)
    r = layer.lin(q, k, v, d, 0.7, h0, starts, do, dht)

    def loss():
        x = layer.lin(q, k, v, d, 0.7, h0, starts)
        return np.sum(x["o"] * do) + np.sum(x["ht"] * dht)

    for name, x in (("dq", q), ("dk", k), ("dv", v), ("dh0", h0)):
        close(r[name], numeric(loss, x))


def test_lin_is_masked_attention():
    """o_i = scale sum_{j <= i} exp(decay (i - j)) (q_i k_j) v_j, one formula without a state."""
    rng = np.random.default_rng(2)
    T, K, V = 9, 4, 3
    q, k, v = rng.normal(size=(T, 1, K)), rng.normal(size=(T, 1, K)), rng.normal(size=(T, 1, V))
    i = np.arange(T)
    m = np.where(i[:, None] >= i, np.exp(-0.4 * (i[:, None] - i)), 0.0)
    want = 0.5 * ((q[:, 0] @ k[:, 0].T) * m) @ v[:, 0]
    got = layer.lin(q, k, v, np.array([-0.4]), 0.5, None, [0, T])
    close(got["o"][:, 0], want)
    one = layer.lin(q, k, v, np.array([-np.inf]), 0.5, None, [0, T])["o"][:, 0]      # every token alone
    close(one, 0.5 * np.sum(q[:, 0] * k[:, 0], 1, keepdims=True) * v[:, 0])


def test_lin_split_calls():
    rng = np.random.default_rng(3)
    q, k, v = (rng.normal(size=(8, 2, 3)) for _ in range(3))
    d = np.array([-0.2, -0.9])
    whole = layer.lin(q, k, v, d, 1.0, None, [0, 8])
    a = layer.lin(q[:5], k[:5], v[:5], d, 1.0, None, [0, 5])
    b = layer.lin(q[5:], k[5:], v[5:], d, 1.0, a["ht"], [0, 3])
    close(np.concatenate([a["o"], b["o"]]), whole["o"])
    close(b["ht"], whole["ht"])


def test_e4m3_table_is_the_formats():
    bits = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    want = np.unique(bits[np.isfinite(bits)])
    assert np.array_equal(layer.e4m3_values(), want)


def test_quant8_keeps_what_it_can_hold():
    rng = np.random.default_rng(4)
    q0 = rng.choice(layer.e4m3_values(), size=(130, 200))
    q0[:, 0] = q0[:, 128] = 448.0
    x = q0 * 0.5
    for rows in (1, 128):
        q, scale, _ = layer.quant8(x, rows)
        assert np.array_equal(q, q0) and np.all(scale == 0.5)
    q, scale, _ = layer.quant8(np.zeros((3, 5)), 1)
    assert not q.any() and not scale.any()


def test_mm8_is_the_product_of_what_the_values_stand_for():
    rng = np.random.default_rng(5)
    a, b = rng.normal(size=(3, 300)), rng.normal(size=(140, 300))
    sa, sb = rng.random((3, 3)), rng.random((2, 3))
    want = np.zeros((3, 140))
    for m in range(3):
        for n in range(140):
            for c in range(300):
                want[m, n] += a[m, c] * sa[m, c // 128] * b[n, c] * sb[n // 128, c // 128]
    close(layer.mm8(a, sa, b, sb), want)
    close(layer.mm8(a, sa, b, np.repeat(sb, 128, 0)[:140]), want)
