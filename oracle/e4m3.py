"""8-bit floating-point rows and weights with power-of-two block scales, and their
products, in fp64 numpy from their definitions.  Codes are bytes; a scale 2^e is the
byte e + 127 (255: NaN)."""
from __future__ import annotations

import numpy as np

BLOCK = 128
TOP = 448.0
EXP = (-100, 120)


def _value(byte: int) -> float:
    sign = -1.0 if byte & 0x80 else 1.0
    exponent, mantissa = (byte >> 3) & 15, byte & 7
    if exponent == 15 and mantissa == 7:
        return float("nan")
    if exponent == 0:
        return sign * mantissa * 2.0 ** -9
    return sign * (1 + mantissa / 8) * 2.0 ** (exponent - 7)


VALUES = np.array([_value(b) for b in range(256)])


def scale_values(byte: np.ndarray) -> np.ndarray:
    """2^(byte - 127) as fp64 (255: NaN)."""
    b = np.asarray(byte, np.int64)
    return np.where(b == 255, np.nan, np.ldexp(1.0, np.where(b == 255, 0, b - 127)))


def rows_values(codes: np.ndarray, scale: np.ndarray) -> np.ndarray:
    """Rows [M, K] from codes and scales [M, blocks]."""
    K = codes.shape[1]
    return VALUES[codes] * np.repeat(scale_values(scale), BLOCK, 1)[:, :K]


def weight_values(codes: np.ndarray, scale: np.ndarray) -> np.ndarray:
    """Weights [N, K] from codes and scales [N blocks, K blocks]."""
    N, K = codes.shape
    return VALUES[codes] * np.repeat(np.repeat(scale_values(scale), BLOCK, 0)[:N], BLOCK, 1)[:, :K]


def exponent(block: np.ndarray) -> int:
    """The exponent of a block's scale: its largest finite magnitude decides."""
    a = np.abs(block[np.isfinite(block)])
    top = a.max() if a.size else 0.0
    e = EXP[0]
    while e < EXP[1] and top > TOP * 2.0 ** e:
        e += 1
    return e


def rows_exponents(x: np.ndarray) -> np.ndarray:
    return np.array([[exponent(row[i:i + BLOCK]) for i in range(0, x.shape[1], BLOCK)] for row in x])


def weight_exponents(w: np.ndarray) -> np.ndarray:
    N, K = w.shape
    return np.array([[exponent(w[n:n + BLOCK, k:k + BLOCK]) for k in range(0, K, BLOCK)] for n in range(0, N, BLOCK)])


def half_step(q: np.ndarray) -> np.ndarray:
    """Half the distance between neighbouring codes at magnitude |q| (at most 448)."""
    a = np.maximum(np.abs(q), 2.0 ** -6)
    return 2.0 ** (np.floor(np.log2(a)) - 4)


def norm(x: np.ndarray, g: np.ndarray, eps: float) -> np.ndarray:
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * g


def silu(z: np.ndarray) -> np.ndarray:
    return z / (1 + np.exp(-z))
