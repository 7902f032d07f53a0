"""CPU oracle of linears in 4 bits with group scales, in float64 with the
roundings of the definition done one by one (numpy's float32 and float16
operations round once, to nearest even)."""
from __future__ import annotations

import numpy as np

GROUP = 128


def encode(W: np.ndarray, zeros: bool):
    """fp32 W [out][in] -> (codes uint8 [out][in], scales uint16 bits [out][T],
    zero points uint8 [out][T]); codes one a byte."""
    out, inf = W.shape
    T = -(-inf // GROUP)
    codes = np.zeros((out, inf), np.uint8)
    scales = np.zeros((out, T), np.float16)
    points = np.full((out, T), 8, np.uint8)
    for t in range(T):
        b = W[:, t * GROUP:(t + 1) * GROUP]
        bad = ~np.isfinite(b).all(1)
        v = np.where(bad[:, None], np.float32(0), b).astype(np.float32)
        with np.errstate(over="ignore"):
            if zeros:
                lo, hi = np.minimum(v.min(1), np.float32(0)), np.maximum(v.max(1), np.float32(0))
                want = (hi - lo) / np.float32(15)
            else:
                want = np.abs(v).max(1) / np.float32(7)
        s16 = np.clip(want, np.float32(2.0 ** -24), np.float32(65504)).astype(np.float16)
        s = s16.astype(np.float32)
        z = np.minimum(np.rint(-lo / s), np.float32(15)) if zeros else np.full(out, 8, np.float32)
        c = np.clip(np.rint(v / s[:, None]) + z[:, None], 0, 15)
        codes[:, t * GROUP:(t + 1) * GROUP] = np.where(bad[:, None], 0, c).astype(np.uint8)
        scales[:, t] = np.where(bad, np.float16(np.nan), s16)
        points[:, t] = np.where(bad & zeros, 0, z).astype(np.uint8)
    return codes, scales.view(np.uint16), points


def pack(codes: np.ndarray) -> np.ndarray:
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack(packed: np.ndarray) -> np.ndarray:
    c = np.empty((packed.shape[0], 2 * packed.shape[1]), np.uint8)
    c[:, 0::2], c[:, 1::2] = packed & 15, packed >> 4
    return c


def values(codes: np.ndarray, scales: np.ndarray, points: np.ndarray) -> np.ndarray:
    """float64 weights [out][in]."""
    inf = codes.shape[1]
    over = (lambda v: np.repeat(v.astype(np.float64), GROUP, 1)[:, :inf])
    return (codes.astype(np.float64) - over(points)) * over(scales.view(np.float16))


def gemm(codes, scales, points, X):
    """(Y [M][out], S [M][out]: the sums of the magnitudes of the terms) of fp16
    bits X [M][in]."""
    w = values(codes, scales, points)
    x = X.view(np.float16).astype(np.float64)
    return x @ w.T, np.abs(x) @ np.abs(w).T
