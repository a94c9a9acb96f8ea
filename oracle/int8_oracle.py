"""CPU oracle of the 8-bit rows (weights and tokens), their product and the
gradient norm.  TEST INFRASTRUCTURE ONLY, like ``lbq_oracle``.

fp32 steps are single numpy float32 operations (one IEEE operation each); the
integer sums are formed in fp64, where sums of products of 8-bit codes over any
row length used here are exact.
"""
from __future__ import annotations

import math

import numpy as np

from .lbq_oracle import bf16_bits, bf16_to_f64

F32 = np.float32


def quantize_rows(x):
    """(codes int8, scales fp32) of the rows of x (fp32 values)."""
    x = np.asarray(x, dtype=F32)
    with np.errstate(all="ignore"):
        top = np.max(np.abs(x), axis=1)
        s = (top / F32(127)).astype(F32)
        s = np.where(s == 0, F32(1), s).astype(F32)
        q = np.clip(np.rint((x / s[:, None]).astype(F32)), -127, 127)
    bad = ~np.isfinite(x).all(axis=1)
    s[bad] = np.nan
    q[bad] = 0
    return q.astype(np.int8), s


def dequant_bf16(codes, scales):
    """bf16 bits of fl(q * s)."""
    return bf16_bits((codes.astype(F32) * scales.astype(F32)[:, None]).astype(F32))


def product(xq, xs, wq, ws):
    """fp32 values fl(fl(fl(acc) * xs) * ws) of the product, before bf16."""
    acc = xq.astype(np.float64) @ wq.astype(np.float64).T
    assert np.abs(acc).max(initial=0) < 2 ** 31
    with np.errstate(all="ignore"):
        y = (acc.astype(F32) * xs.astype(F32)[:, None]).astype(F32)
        return (y * ws.astype(F32)[None, :]).astype(F32)


def product_bf16(xq, xs, wq, ws):
    return bf16_bits(product(xq, xs, wq, ws))


def tokens(x_bits):
    """Codes and scales of bf16 tokens (bit patterns)."""
    return quantize_rows(bf16_to_f64(x_bits).astype(F32))


def grad_norm(tensors, kind="2"):
    """Norm in fp64 over arrays of exact values."""
    flat = [np.asarray(t, dtype=np.float64).ravel() for t in tensors]
    if kind == "inf":
        return max((float(np.max(np.abs(t))) for t in flat if t.size), default=0.0)
    return math.sqrt(math.fsum(float(v) * float(v) for t in flat for v in t))


def clip_factor(norm, max_norm):
    return min(1.0, max_norm / (norm + 1e-6))
