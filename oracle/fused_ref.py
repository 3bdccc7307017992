"""NumPy oracle of the RMS norm with 8-bit outputs, of the fused epilogues and of the BF16
products. TEST INFRASTRUCTURE ONLY: only ``tests/`` may import it. It shares no code or
tables with the HIP library.

The norm, the activations and the BF16 products are this library's own definitions
(parity unpinned by the pages); the quantizers behind the norm are the oracle's own.

  norm   h = BF16(fl32(x + residual)) or x; r = fl32(1 / sqrt(sum h^2 / K + eps)) in
         float64 up to the last rounding; n = fl32(fl32(h r) w)
  act    float64: relu, silu, gelu (v Phi(v)), gelu_tanh; swiglu of [gate | up] columns
  product64 / linear64: float64 sums
"""

from __future__ import annotations

import math

import numpy as np

from .w8a8_ref import bf16_to_f32, f32_to_bf16

__all__ = ["norm", "act64", "swiglu64", "product64", "ACTS"]

ACTS = ("none", "swiglu", "relu", "silu", "gelu", "gelu_tanh")


def norm(x_bits, w_bits=None, eps: float = 1e-6, residual_bits=None):
    """BF16 bits [M, K] (and [K], [M, K]) -> (h bits [M, K], n float32 [M, K])."""
    h = np.asarray(x_bits)
    if residual_bits is not None:
        h = f32_to_bf16((bf16_to_f32(x_bits) + bf16_to_f32(residual_bits)).astype(np.float32))
    v = bf16_to_f32(h)
    wide = v.astype(np.float64)
    r = (1.0 / np.sqrt((wide * wide).sum(1) / v.shape[1] + eps)).astype(np.float32)
    n = (v * r[:, None]).astype(np.float32)
    if w_bits is not None:
        n = (n * bf16_to_f32(w_bits)[None]).astype(np.float32)
    return h, n


_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def _sigmoid(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def act64(v, act: str):
    """float64 activation of float64 values."""
    v = np.asarray(v, np.float64)
    if act == "relu":
        return np.maximum(v, 0.0)
    if act == "silu":
        return v * _sigmoid(v)
    if act == "gelu":
        return 0.5 * v * _erfc(-v / math.sqrt(2.0))
    if act == "gelu_tanh":
        return v * _sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3))
    return v


def swiglu64(v):
    """float64 [M, 2 I] = [gate | up] -> silu(gate) up."""
    half = v.shape[1] // 2
    return act64(v[:, :half], "silu") * v[:, half:]


def product64(x_bits, w_bits):
    """(sum_k x w, sum_k |x w|) in float64."""
    x, w = bf16_to_f32(x_bits).astype(np.float64), bf16_to_f32(w_bits).astype(np.float64)
    return x @ w.T, np.abs(x) @ np.abs(w).T
