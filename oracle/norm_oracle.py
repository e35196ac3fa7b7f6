"""Residual addition, root-mean-square norm, rotation and int8 quantization of
activation rows: the plain CPU oracle.

TEST INFRASTRUCTURE.  Only tests/ and __graft_entry__.smoke() may import this
module; the HIP library shares no code with it.

  N1. h = x + residual in fp32 (one rounding); it becomes the residual.
  N2. r = 1 / sqrt(sum h^2 / K + eps) in fp64, rounded once to fp32.
  N3. u = (h * r) * weight, two fp32 roundings.
  N4. u is rotated and quantized as any activation row (svg_oracle.quant_acts).
`norm_f64` is the same norm with no rounding but fp64's.
"""
import numpy as np

from . import svg_oracle as O


def norm_rows(x, residual, weight, eps):
    """(h, u) of N1-N3: fp32 rows, every step rounded as the definition says."""
    f = np.float32
    h = x.astype(f) if residual is None else x.astype(f) + residual.astype(f)
    K = h.shape[1]
    r = (1.0 / np.sqrt((h.astype(np.float64) ** 2).sum(1) / K + eps)).astype(f)
    return h, (h * r[:, None]) * weight.astype(f)


def norm_quant(x, residual, weight, eps, signs, block):
    """(h, u, codes [M, K] int8, scales [M] fp32)."""
    h, u = norm_rows(x, residual, weight, eps)
    q, s = O.quant_acts(u, signs, block)
    return h, u, q, s


def norm_f64(x, residual, weight, eps):
    h = x.astype(np.float64) + (0 if residual is None else residual.astype(np.float64))
    return h / np.sqrt((h ** 2).mean(1, keepdims=True) + eps) * weight.astype(np.float64)


def slab_codes(q):
    """Row-major codes [M, K] as the slab buffers of 32 rows that follow one
    another: the code of (row m, k) of a buffer of R rows is byte
    ((k / 32) * R + m % 32) * 32 + k % 32 of it."""
    M, K = q.shape
    out = np.empty(M * K, np.int8)
    for b in range(0, M, 32):
        R = min(32, M - b)
        part = out[b * K:(b + R) * K]
        for m in range(R):
            for k0 in range(0, K, 32):
                at = ((k0 // 32) * R + m) * 32
                part[at:at + 32] = q[b + m, k0:k0 + 32]
    return out
