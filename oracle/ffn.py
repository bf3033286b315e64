"""Gradients of the gated feed-forward block and of the combine, and low-rank
adapters.  ORACLE (test infrastructure only).

  block    z = x W', h = silu(z_g) z_u with z_g, z_u the halves of z's columns
  swiglu_grad   dz_g = dh z_u silu'(z_g), dz_u = dh silu(z_g),
           silu'(g) = s (1 + g (1 - s)), s = sigmoid(g)
  combine  out[t] = sum_j w[t, j] y[inv[t, j]]
  combine_grad  dy[inv[i]] = w[i] dout[i // k], dw[i] = <dout[i // k], y[inv[i]]>
  lora     base + scale[a] (x a_a') b_a' of each row's adapter a

Plain float64.
"""
from __future__ import annotations

import numpy as np


def _sigmoid(g):
    return 1.0 / (1.0 + np.exp(-g))


def swiglu_grad(dh, z):
    z, dh = np.asarray(z, np.float64), np.asarray(dh, np.float64)
    H = z.shape[1] // 2
    g, u, s = z[:, :H], z[:, H:], _sigmoid(z[:, :H])
    return np.concatenate([dh * u * s * (1.0 + g * (1.0 - s)), dh * g * s], axis=1)


def combine_grad(dout, y, inv_perm, w, k: int):
    """(dy, dw); rows of dy that no entry of inv_perm names are NaN."""
    dout, y, w = (np.asarray(a, np.float64) for a in (dout, y, w))
    dy, dw = np.full_like(y, np.nan), np.zeros(len(w))
    for i, r in enumerate(inv_perm):
        if 0 <= r < len(y):
            dy[r] = w[i] * dout[i // k]
            dw[i] = dout[i // k] @ y[r]
    return dy, dw


def lora(x, a, b, scale, ids, base, slices: int = 1):
    """The projection with its adapters, before an epilogue: [T, N]."""
    x, a, b, scale = (np.asarray(v, np.float64) for v in (x, a, b, scale))
    N, rank = b.shape[1:]
    n = N // slices
    y = np.array(base, np.float64)
    for t, e in enumerate(ids):
        if 0 <= e < len(a):
            v = a[e] @ x[t]
            for s in range(slices):
                y[t, s * n:(s + 1) * n] += scale[e] * (b[e, s * n:(s + 1) * n] @ v[s * rank:(s + 1) * rank])
    return y
