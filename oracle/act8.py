"""Activation checkpoints in 8 bits, for the oracle.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Blocks of 64 values along a row: a = max |x|, code = the exact quotient
127 x / a rounded half to even, scale = a / 127 rounded to float32; a block of
zeros has codes and scale 0, a block with an infinity or a NaN codes 0 and
scale NaN.  In float64, 127 x (15 significant bits for a bf16 x) divided by an
8-bit a is never within rounding of a half-integer unless it is one, so
numpy's rint of the float64 quotient is the exact rounding.
"""
import numpy as np

BLOCK = 64


def quantize(x):
    """(codes int8 [rows, cols], scale float32 [cols / 64, rows up to 32]) of
    the float64 values x [rows, cols] of bf16 activations."""
    rows, cols = x.shape
    b = np.asarray(x, dtype=np.float64).reshape(rows, cols // BLOCK, BLOCK)
    with np.errstate(invalid="ignore"):
        a = np.abs(b).max(axis=2)
        ok = np.isfinite(b).all(axis=2)
        div = np.where(ok & (a > 0), a, 1.0)[..., None]
        codes = np.where((ok & (a > 0))[..., None], np.rint(127.0 * b / div), 0.0)
    scale = np.zeros((cols // BLOCK, (rows + 31) // 32 * 32), dtype=np.float32)
    scale[:, :rows] = np.where(ok, np.where(ok, a, 0.0).astype(np.float32) / np.float32(127),
                               np.float32(np.nan)).T
    return codes.astype(np.int8).reshape(rows, cols), scale


def dequantize(codes, scale):
    """float32 values fl(code * scale) [rows, cols]."""
    rows, cols = codes.shape
    c = codes.astype(np.float32).reshape(rows, cols // BLOCK, BLOCK)
    return (c * scale[:, :rows].T[..., None]).reshape(rows, cols)
