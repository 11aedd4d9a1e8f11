"""Root-mean-square norm with the residual's addition, and rows to int8, float64.

The norm in front of the LM head; the DFlash 2 pages publish no counterpart.
h = bf16(x + residual) (the sum of two bf16 values, rounded to nearest even),
y = h gamma / sqrt(mean h^2 + eps).  The int8 form gives q = rint(127 p / a)
and scale = a r / 127 with p = h gamma, a = max |p|, r = 1 / sqrt(mean h^2 +
eps).  p has at most 16 significant bits, so 127 p and a are exact in float64
and the correctly rounded quotient is a half only where the real one is.
"""
import numpy as np

from ._widen import bf16


def round_bf16(a) -> np.ndarray:
    """float64 -> nearest bf16 value (ties to even) as float64; finite inputs
    whose magnitude is a normal bf16's."""
    a = np.asarray(a, dtype=np.float64)
    m, e = np.frexp(a)
    return np.ldexp(np.rint(np.ldexp(m, 8)), e - 8)


def residual_sum(x_bits, residual_bits=None) -> np.ndarray:
    x = bf16(x_bits)
    return x if residual_bits is None else round_bf16(x + bf16(residual_bits))


def rmsnorm(x_bits, gamma_bits, residual_bits=None, eps=1e-6):
    """(y, h, r), float64; y is not rounded."""
    h = residual_sum(x_bits, residual_bits)
    r = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    return h * bf16(gamma_bits) * r[:, None], h, r


def quantise(p: np.ndarray, r=1.0):
    """Rows p (exact products) -> (q int8, scale float64)."""
    a = np.abs(p).max(axis=1)
    live = a >= 2.0 ** -100
    safe = np.where(live, a, 1.0)
    q = np.where(live[:, None], np.rint(127.0 * p / safe[:, None]), 0.0)
    return q.astype(np.int8), np.where(live, a * r / 127.0, 0.0)


def rmsnorm_i8(x_bits, gamma_bits, residual_bits=None, eps=1e-6):
    """(q, scale, h)."""
    _, h, r = rmsnorm(x_bits, gamma_bits, residual_bits, eps)
    q, scale = quantise(h * bf16(gamma_bits), r)
    return q, scale, h


def quant_i8(x_bits):
    return quantise(bf16(x_bits))
