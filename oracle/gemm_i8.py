"""Int8 matrix product with a scale per token and per channel.

C[m,n] = f32(f32(f32(sum_k A[m,k] B[n,k]) * sa[m]) * sb[n]): the integer sum
is exact and the three roundings to fp32 are part of the definition, so the
result is a value, not an interval.  The DFlash 2 pages have no counterpart.
"""
import numpy as np


def product(A, B) -> np.ndarray:
    """Exact integer sums, int64.  Sums of int8 products of K <= 131071 are
    below 2^31 and every partial sum is exact in float64, so the product may
    run in floating point."""
    return np.rint(A.astype(np.float64) @ B.astype(np.float64).T).astype(np.int64)


def gemm_i8(A, sa, B, sb) -> np.ndarray:
    c = product(A, B).astype(np.float32)
    return c * sa.astype(np.float32)[:, None] * sb.astype(np.float32)[None, :]
