"""CPU oracle of linears in 8-bit floating point blocks of 128 and of 8-bit
activation checkpoints, in float64 with table look-ups.

Written from the definitions and nothing else: the codes of a format come
from a sorted table of every value the format has, so no arithmetic is
shared with the kernels (which scale, convert and repair in fp32).
"""
from __future__ import annotations

import numpy as np

BLOCK = 128
TINY = 2.0 ** -100


def e4m3_table() -> np.ndarray:
    """float64 value of each of the 256 OCP e4m3 codes (1 sign, 4 exponent
    bits with bias 7, 3 fraction bits; no infinities, NaN at 0x7F and 0xFF)."""
    v = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        m = f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
        v[c] = np.nan if (c & 0x7F) == 0x7F else (-m if c & 0x80 else m)
    return v


_E4M3 = e4m3_table()
_POS = _E4M3[:0x7F]                       # 0 .. 448, ascending
_F16_POS = np.arange(0x7C00, dtype=np.uint16).view(np.float16).astype(np.float64)   # 0 .. 65504, ascending


def _nearest(table: np.ndarray, v: np.ndarray) -> np.ndarray:
    """Index of the entry of an ascending table nearest to v >= 0 (v at most
    the last entry), ties to the even index: codes of one sign are consecutive
    and an even code has an even significand."""
    hi = np.clip(np.searchsorted(table, v), 1, len(table) - 1)
    lo = hi - 1
    dl, dh = v - table[lo], table[hi] - v
    return np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)


def e4m3_codes(v: np.ndarray) -> np.ndarray:
    """Codes of float64 v, |v| <= 448 (or rounding to it)."""
    mag = np.minimum(np.abs(v), 448.0)
    return (_nearest(_POS, mag) | np.where(np.signbit(v), 0x80, 0)).astype(np.uint8)


def e4m3_values(codes: np.ndarray) -> np.ndarray:
    return _E4M3[codes]


def _block(v: np.ndarray):
    """(codes, scale fp32) of one block of float64 values."""
    if not np.isfinite(v).all():
        return np.zeros(v.shape, np.uint8), np.float32(np.nan)
    A = max(float(np.abs(v).max(initial=0.0)), TINY)
    inv = float(np.float32(448.0 / A))
    return e4m3_codes((v * inv).astype(np.float32).astype(np.float64)), np.float32(A / 448.0)


def _slices(n: int):
    return [slice(i, min(n, i + BLOCK)) for i in range(0, n, BLOCK)]


def encode(W: np.ndarray):
    """fp32 W [out][in] -> (codes uint8, scales fp32 [ceil(out/128)][T])."""
    out, inf = W.shape
    codes = np.zeros((out, inf), np.uint8)
    scales = np.zeros((len(_slices(out)), len(_slices(inf))), np.float32)
    for i, r in enumerate(_slices(out)):
        for t, c in enumerate(_slices(inf)):
            codes[r, c], scales[i, t] = _block(W[r, c].astype(np.float64))
    return codes, scales


def quantize(X: np.ndarray):
    """fp16 bits [M][in] -> (codes uint8, scales fp32 [T][M])."""
    M, inf = X.shape
    x = X.view(np.float16).astype(np.float64)
    codes = np.zeros((M, inf), np.uint8)
    scales = np.zeros((len(_slices(inf)), M), np.float32)
    for m in range(M):
        for t, c in enumerate(_slices(inf)):
            codes[m, c], scales[t, m] = _block(x[m, c])
    return codes, scales


def values(codes: np.ndarray, scales: np.ndarray, rows: int) -> np.ndarray:
    """float64 values of codes [n][in] with scales [..][T] per `rows` rows."""
    s = np.repeat(np.repeat(scales.astype(np.float64), BLOCK, 1)[:, :codes.shape[1]], rows, 0)[:codes.shape[0]]
    return e4m3_values(codes) * s


def gemm(codes, scales, x_codes, x_scales):
    """(Y, sum of the magnitudes of its terms), float64 [M][out]."""
    w = values(codes, scales, BLOCK)
    x = values(x_codes, np.ascontiguousarray(x_scales.T), 1)
    return x @ w.T, np.abs(x) @ np.abs(w).T


def largest_products(codes, scales, x_codes, x_scales):
    """Sum over the groups of 8 columns of the largest |x w| of a group,
    float64 [M][out]."""
    w = np.abs(values(codes, scales, BLOCK))
    x = np.abs(values(x_codes, np.ascontiguousarray(x_scales.T), 1))
    total = np.zeros((x.shape[0], w.shape[0]))
    for c in range(0, w.shape[1], 8):
        top = np.zeros_like(total)
        for j in range(c, c + 8):
            np.maximum(top, np.outer(x[:, j], w[:, j]), out=top)
        total += top
    return total


def checkpoint(X: np.ndarray):
    """fp16 bits [M][in] -> (codes int8 [M][in], scale bits uint16 [M][T])."""
    M, inf = X.shape
    x = X.view(np.float16).astype(np.float64)
    codes = np.zeros((M, inf), np.int8)
    scales = np.zeros((M, len(_slices(inf))), np.uint16)
    for t, c in enumerate(_slices(inf)):
        for m in range(M):
            v = x[m, c]
            if not np.isfinite(v).all():
                scales[m, t] = 0x7E00
                continue
            bits = int(np.searchsorted(_F16_POS, np.abs(v).max() / 127.0))   # smallest fp16 not below it
            bits = min(max(bits, 1), int(np.searchsorted(_F16_POS, 515.5)))
            scales[m, t] = bits
            codes[m, c] = np.clip(np.rint(v / _F16_POS[bits]), -127, 127).astype(np.int8)
    return codes, scales


def restore(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """fp16 bits [M][in] of the values a checkpoint stands for."""
    s = np.repeat(scales.view(np.float16).astype(np.float64), BLOCK, 1)[:, :codes.shape[1]]
    return (codes.astype(np.float64) * s).astype(np.float16).view(np.uint16)
