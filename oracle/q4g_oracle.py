"""Oracle of the matrix-vector products with 4-bit weights and group scales, float64 numpy from the
definition: w = s (v - z), y = act(x w^T + bias) + residual."""
from __future__ import annotations

import numpy as np


def values(w):
    """v int [N, K] of packed bytes [N, K/2], the even value in the low four bits."""
    w = np.asarray(w, np.uint8)
    v = np.empty((w.shape[0], 2 * w.shape[1]), np.int64)
    v[:, 0::2], v[:, 1::2] = w & 15, w >> 4
    return v


def product(x, w, scales, zeros, group: int, offset: float = 0.0):
    """(x w^T, T) float64 [M, N]; T = sum_k |x s| (offset + v + |offset + z|), the absolute values of the
    terms that a sum is made of which takes s (sum x (offset + v) - (offset + z) sum x)."""
    x = np.asarray(x, np.float64)
    v = values(w)
    M, K = x.shape
    y, T = np.zeros((M, v.shape[0])), np.zeros((M, v.shape[0]))
    for g, k0 in enumerate(range(0, K, group)):
        s = np.asarray(scales, np.float64)[:, g]
        z = 8.0 if zeros is None else np.asarray(zeros, np.float64)[:, g:g + 1]
        part, vg = x[:, k0:k0 + group], v[:, k0:k0 + group]
        y += (part @ (vg - z).T) * s
        T += (np.abs(part) @ (offset + vg + np.abs(offset + z)).T) * np.abs(s)
    return y, T


def bound(T, K: int):
    """How far a float32 evaluation may be off. A result's longest chain of additions: the 128 products
    of a record on the matrix unit, whose additions are taken to be good to a whole unit in the last
    place (2^-23), 3 pieces, the zero and the scale, at most 4 folds for each of the K/128 records and 16
    wavefronts, half a unit (2^-24) each."""
    records = -(-K // 128)
    return (2 * 128 + 2 + 4 * records + 16 + 3) * 2.0 ** -24 * T
