"""Microscaled (MX) rows and their product.  ORACLE (test infrastructure
only).

Blocks of 32 consecutive elements share one power-of-two scale (E8M0: byte s
stands for 2^(s-127), 255 for NaN); elements are E2M1 ("mxfp4") or E4M3
("mxfp8").  Quantization of a block with largest magnitude amax:

  s    = clamp(127 + floor(log2 amax) - emax, 0, 254), emax = 2 (E2M1) or
         8 (E4M3); 0 when amax = 0
  code = element nearest to x / 2^(s-127), ties to the even code, saturating;
         zero is +0
  a block with an infinity or a NaN: s = 255, codes 0

Everything is exact in float64: x is fp32 or bf16, the quotient a power-of-two
multiple of it.
"""
from __future__ import annotations

import numpy as np

from .formats import E2M1_VALUES, E4M3_VALUES, bf16_round, e2m1_encode, e4m3_encode

EMAX = {"mxfp4": 2, "mxfp8": 8}


def mx_quantize(x, fmt: str):
    """[rows, K] finite or not -> (codes uint8, scales uint8 [rows, K/32])."""
    x = np.asarray(x, np.float64)
    rows, K = x.shape
    if K % 32:
        raise ValueError("K must be a multiple of 32")
    b = x.reshape(rows, K // 32, 32)
    bad = ~np.isfinite(b).all(axis=2)
    b = np.where(bad[:, :, None], 0.0, b)
    amax = np.abs(b).max(axis=2)
    _, e = np.frexp(amax)                         # amax = m 2^e, m in [0.5, 1)
    s = np.clip(127 + (e - 1) - EMAX[fmt], 0, 254)
    s = np.where(amax > 0, s, 0)
    q = np.ldexp(b, -(s - 127)[:, :, None])
    if fmt == "mxfp4":
        c = e2m1_encode(q).reshape(rows, K)
        codes = (c[:, 0::2] | (c[:, 1::2] << 4)).astype(np.uint8)
    else:
        mag = e4m3_encode(np.abs(q))
        codes = (mag | (((q < 0) & (mag != 0)).astype(np.uint8) << 7)).reshape(rows, K)
    return codes, np.where(bad, 255, s).astype(np.uint8)


def mx_decode(codes, scales, fmt: str) -> np.ndarray:
    """float64 values of MX rows; NaN where the scale is 255."""
    codes, scales = np.asarray(codes), np.asarray(scales)
    if fmt == "mxfp4":
        v = np.empty(codes.shape[:-1] + (codes.shape[-1] * 2,))
        v[..., 0::2], v[..., 1::2] = E2M1_VALUES[codes & 15], E2M1_VALUES[codes >> 4]
    else:
        v = E4M3_VALUES[codes]
    f = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return v * np.repeat(f, 32, axis=-1)


def mx_gemm(x_rows, W) -> np.ndarray:
    """Decoded rows [m, K] times decoded W^T [N, K], float64."""
    return np.asarray(x_rows, np.float64) @ np.asarray(W, np.float64).T


def rmsnorm(x, weight, eps: float, residual=None):
    """(s, y before its bf16 rounding) in float64: s = bf16(x + residual), or x;
    y = s / sqrt(mean(s^2) + eps) * weight."""
    s = np.asarray(x, np.float64)
    if residual is not None:
        s = bf16_round(s + np.asarray(residual, np.float64))
    r = 1.0 / np.sqrt((s * s).mean(axis=1, keepdims=True) + eps)
    return s, s * r * np.asarray(weight, np.float64)
