"""Bounds of a q4_G product with one value that is not 0 in each token, scale 1 and whole zeros."""
import numpy as np


def one_value_bound(x, v, z):
    """How far x (v - z) may be off for a float32 x, float64 arrays. The kernel adds the products p (16 +
    v) of x's three pieces p, which are exact (8 and 5 bits), the two smaller of them exactly (within 21
    bits): one rounding of x (16 + v), half a unit. The sum of the pieces is x, exactly, and one more
    rounding takes (16 + z) x off: half a unit of x (v - z). The rest adds zeros. (1 + 2^-20: units are
    relative to the rounded values.)"""
    x, v, z = (np.asarray(a, np.float64) for a in (x, v, z))
    return 2.0 ** -24 * np.abs(x) * (16 + v + np.abs(v - z)) * (1 + 2.0 ** -20)


def full_mantissas(n, seed):
    """n float32 values in +-[1, 2) of 24 significant bits whose three pieces have 8 each: bit 15 is
    set, and the last eight bits are 193 to 255."""
    rng = np.random.default_rng(seed)
    m = ((1 << 23) + (rng.integers(0, 128, n) << 16) + ((128 + rng.integers(0, 128, n)) << 8)
         + 193 + 2 * rng.integers(0, 32, n))
    return (m * 2.0 ** -23 * rng.choice((-1.0, 1.0), n)).astype(np.float32)
