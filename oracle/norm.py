"""RMSNorm around a block, forward and backward (CPU oracle).

TEST INFRASTRUCTURE ONLY -- see the package docstring.

  n = x r w with r = (mean x^2 + eps)^(-1/2), rounded once to BF16. Everything up to that
  rounding is done in 80-bit extended precision (relative error below 2^-60), so the BF16
  value is the correctly rounded one unless the exact value lies that close to a midpoint.
  out = res_scale x + branch_scale gate (y r w).
  Gradients in FP64 from their formulas: g = dn w, xh = x r,
  dx = r (g - xh mean(g xh)) + res_scale d_res, dw = sum over rows of dn xh.
"""

from __future__ import annotations

import numpy as np

LD = np.longdouble


def _bf16_bits_from_extended(v) -> np.ndarray:
    """Extended-precision values to BF16 bits, one rounding, to nearest even (normal range and
    zero; |v| < 2^-126 is rounded on the subnormal grid, overflow gives infinity)."""
    v = np.asarray(v, dtype=LD)
    m, e = np.frexp(np.abs(v))                                # |v| = m 2^e, m in [0.5, 1)
    e = np.maximum(e, -125)                                   # subnormal grid below 2^-126
    quantum = np.ldexp(LD(1), e - 8)
    q = np.rint(np.abs(v) / quantum) * quantum                # both steps exact but the rounding
    with np.errstate(over="ignore"):
        f = np.copysign(q, v).astype(np.float32)              # exact
    return (f.view(np.uint32) >> np.uint32(16)).astype(np.uint16)


def rstd(x, eps: float) -> np.ndarray:
    """(rows,) extended precision."""
    x = np.asarray(x, dtype=LD)
    return LD(1) / np.sqrt(np.mean(x * x, axis=1) + LD(eps))


def rmsnorm_bf16(x, weight, eps: float) -> np.ndarray:
    """BF16 bits of the correctly rounded n; x (rows, cols) float values, weight (cols) or None."""
    x = np.asarray(x, dtype=LD)
    n = x * rstd(x, eps)[:, None]
    if weight is not None:
        n = n * np.asarray(weight, dtype=LD)
    return _bf16_bits_from_extended(n)


def gate_residual(x, y, weight, gate, eps: float, branch_scale: float, res_scale: float) -> np.ndarray:
    """FP64 out; gate broadcast to (rows, cols) by the caller, or None."""
    x, y = np.asarray(x, np.float64), np.asarray(y, np.float64)
    b = y * rstd(y, eps).astype(np.float64)[:, None]
    if weight is not None:
        b = b * np.asarray(weight, np.float64)
    if gate is not None:
        b = b * np.asarray(gate, np.float64)
    return res_scale * x + branch_scale * b


def backward(dn, x, r, weight):
    """FP64 (dx, dw) of n = x r w for the gradient dn of n; r (rows,) as the forward stored it."""
    dn, x = np.asarray(dn, np.float64), np.asarray(x, np.float64)
    r = np.asarray(r, np.float64)[:, None]
    xh = x * r
    g = dn if weight is None else dn * np.asarray(weight, np.float64)
    dx = r * (g - xh * np.mean(g * xh, axis=1, keepdims=True))
    return dx, np.sum(dn * xh, axis=0)
