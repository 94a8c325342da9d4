"""FP64 oracle of the layer operators: short causal convolution, selective state
space scan, root-mean-square norm; forward and hand-derived backward.

TEST INFRASTRUCTURE ONLY (see the package docstring). Plain loops over the
sequences and tokens, vectorised over channels; packed token axis [tokens, ...]
with ``starts`` (N + 1 offsets). Pinned in ``tests/test_oracle_layer.py`` by
finite differences and closed forms.

    conv:  s_t = bias + sum_j w[:, j] x_{t-W+1+j},  y = s or s sigmoid(s)
    scan:  delta = softplus(dt + dt_bias),  a = exp(-delta exp(A_log))
           h_t = a h_{t-1} + delta x_t b_t,  y = (c_t . h_t + d_skip x_t) silu(z_t)
    norm:  h = x + residual,  y = h (mean h^2 + eps)^(-1/2) w
"""

from __future__ import annotations

import numpy as np


def sigmoid(v):
    return 0.5 * (1.0 + np.tanh(0.5 * v))


def softplus(v):
    return np.logaddexp(0.0, v)


def conv(x, w, bias, h0, starts, silu, dy=None, dfinal=None):
    """x [tokens, D], w [D, W], bias [D] or None, h0 [N, W-1, D] or None. Returns a
    dict with y, final and, given dy, dx, dweight, dbias, dinit."""
    D, W = w.shape
    N = len(starts) - 1
    h0 = np.zeros((N, W - 1, D)) if h0 is None else h0
    out = dict(y=np.zeros_like(x), final=np.zeros_like(h0))
    if dy is not None:
        out.update(dx=np.zeros_like(x), dweight=np.zeros_like(w), dbias=np.zeros(D), dinit=np.zeros_like(h0))
    for n in range(N):
        lo, hi = starts[n], starts[n + 1]
        L = hi - lo
        ext = np.concatenate([h0[n], x[lo:hi]])
        out["final"][n] = ext[L:]
        s = sum(w[:, j] * ext[j:j + L] for j in range(W)) + (0.0 if bias is None else bias)
        sg = sigmoid(s)
        out["y"][lo:hi] = s * sg if silu else s
        if dy is None:
            continue
        ds = dy[lo:hi] * (sg * (1.0 + s * (1.0 - sg)) if silu else 1.0)
        dext = np.zeros_like(ext)
        for j in range(W):
            dext[j:j + L] += w[:, j] * ds
            out["dweight"][:, j] += np.sum(ds * ext[j:j + L], axis=0)
        if dfinal is not None:
            dext[L:] += dfinal[n]
        out["dbias"] += ds.sum(axis=0)
        out["dinit"][n] = dext[:W - 1]
        out["dx"][lo:hi] = dext[W - 1:]
    return out


def scan(x, dt, A_log, b, c, d_skip, z, dt_bias, h0, starts, use_softplus=True, dy=None, dht=None):
    """x, dt, z [tokens, D]; b, c [tokens, G, S]; A_log [D, S]; h0 [N, D, S] or
    None. Returns a dict with y, ht and, given dy, every gradient."""
    T, D = x.shape
    G, S = b.shape[1:]
    N, M = len(starts) - 1, D // G
    skip = np.zeros(D) if d_skip is None else d_skip
    raw = dt if dt_bias is None else dt + dt_bias
    delta = softplus(raw) if use_softplus else raw
    A = -np.exp(A_log)
    h0 = np.zeros((N, D, S)) if h0 is None else h0
    out = dict(y=np.zeros_like(x), ht=np.zeros_like(h0))
    if dy is not None:
        out.update(dx=np.zeros_like(x), ddt=np.zeros_like(x), dz=np.zeros_like(x), db=np.zeros_like(b),
                   dc=np.zeros_like(c), dA_log=np.zeros_like(A), dd_skip=np.zeros(D), ddt_bias=np.zeros(D),
                   dh0=np.zeros_like(h0))

    def wide(v):   # [G, S] -> [D, S]
        return np.repeat(v, M, axis=0)

    for n in range(N):
        lo, hi = starts[n], starts[n + 1]
        h = h0[n].copy()
        hs = [h]
        for t in range(lo, hi):
            h = np.exp(delta[t][:, None] * A) * h + (delta[t] * x[t])[:, None] * wide(b[t])
            hs.append(h)
            y0 = np.sum(h * wide(c[t]), axis=1) + skip * x[t]
            out["y"][t] = y0 if z is None else y0 * z[t] * sigmoid(z[t])
        out["ht"][n] = h
        if dy is None:
            continue
        r = np.zeros((D, S)) if dht is None else dht[n].copy()
        for t in range(hi - 1, lo - 1, -1):
            h, hp = hs[t - lo + 1], hs[t - lo]
            B, C = wide(b[t]), wide(c[t])
            a = np.exp(delta[t][:, None] * A)
            d0 = dy[t]
            if z is not None:
                sg = sigmoid(z[t])
                y0 = np.sum(h * C, axis=1) + skip * x[t]
                out["dz"][t] = dy[t] * y0 * sg * (1.0 + z[t] * (1.0 - sg))
                d0 = dy[t] * z[t] * sg
            g = r + C * d0[:, None]
            out["dc"][t] = (h * d0[:, None]).reshape(G, M, S).sum(axis=1)
            out["db"][t] = (g * (delta[t] * x[t])[:, None]).reshape(G, M, S).sum(axis=1)
            s1 = np.sum(g * B, axis=1)
            w = g * a * hp
            out["dx"][t] = delta[t] * s1 + skip * d0
            dd = x[t] * s1 + np.sum(w * A, axis=1)
            out["ddt"][t] = dd * sigmoid(raw[t]) if use_softplus else dd
            out["dA_log"] += w * delta[t][:, None] * A
            out["dd_skip"] += d0 * x[t]
            out["ddt_bias"] += out["ddt"][t]
            r = g * a
        out["dh0"][n] = r
    return out


def norm(x, w, residual, eps, dy=None, dres=None):
    """x [rows, D]. Returns a dict with y, h and, given dy (then x is the stored
    sum and residual None), dx and dweight."""
    h = x if residual is None else x + residual
    r = 1.0 / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
    out = dict(y=h * r * w, h=h)
    if dy is not None:
        u, v = h * r, dy * w
        out["dx"] = r * (v - u * np.mean(u * v, axis=1, keepdims=True)) + (0.0 if dres is None else dres)
        out["dweight"] = np.sum(dy * u, axis=0)
    return out
