"""Oracle linear with 4-bit weights and group scales (test infrastructure only), float64.

``out = sum_k x[m, k] * (q[n, k] - z[n, k // G]) * s[n, k // G] + bias[n]`` with unsigned 4-bit
codes (element 2j in the low nibble of byte j), one scale per group of G elements of a row, zero
points packed like the codes along the groups (8 everywhere when there are none).
"""

import numpy as np


def unpack4(packed: np.ndarray, n: int) -> np.ndarray:
    """uint8 [rows, bytes] -> float64 [rows, n] of its nibbles, low nibble first."""
    p = np.asarray(packed, np.uint8)
    out = np.empty((p.shape[0], p.shape[1] * 2), np.float64)
    out[:, 0::2] = p & 0x0F
    out[:, 1::2] = p >> 4
    return out[:, :n]


def int4_weight(packed, scale, zero, group):
    """The weights [N, K] in float64."""
    K = packed.shape[1] * 2
    q = unpack4(packed, K)
    z = np.full((q.shape[0], K // group), 8.0) if zero is None else unpack4(zero, K // group)
    s = np.asarray(scale, np.float64)
    return (q - np.repeat(z, group, axis=1)) * np.repeat(s, group, axis=1)


def int4_linear(x, packed, scale, zero, group, bias=None):
    """float64 [M, N], not rounded."""
    out = np.asarray(x, np.float64) @ int4_weight(packed, scale, zero, group).T
    return out if bias is None else out + np.asarray(bias, np.float64)[None, :]
