"""Inputs and references of the layer operators' tests."""
import numpy as np

import oracle
import synth
from oracle import layer_oracle as lo

BAR = 1e-5  # the product's own bound, in units of T


def product(x, w):
    """(P, T) float64 of f32 activations and q4_K blocks."""
    q, f = oracle.quantize_q8_1(x), oracle.decode_q4_K(w)
    return oracle.mmq(q, f), oracle.mmq_terms(q, f)[1]


def weights(N, K, seed, kind="fit"):
    return synth.q4k_weights(kind, N, K, seed)[0]


def pair_columns(F):
    """Columns of the gate rows and of the up rows among the packed rows."""
    f = np.arange(F)
    g = 16 * (f // 8) + f % 8
    return g, g + 8


def experts_gated(x, ids, gate, up, act):
    """(H, err) float64 [M*k, F]; NaN rows for pairs without an expert."""
    M, k = ids.shape
    E, F = gate.shape[:2]
    H = np.full((M * k, F), np.nan)
    err = np.zeros((M * k, F))
    for e in range(E):
        ps = np.nonzero(ids.reshape(-1) == e)[0]
        if ps.size:
            rows = np.ascontiguousarray(x[ps // k])
            (G, TG), (U, TU) = product(rows, gate[e]), product(rows, up[e])
            H[ps], err[ps] = lo.gated(G, TG, U, TU, BAR, act)
    return H, err


def experts_down(H, ids, wts, down, residual):
    """(out, err) float64 [M, D]. Beside the product's bar each of the at most k*F/256 super-block
    contributions is scaled and added in float32, and up to 16 wavefronts' sums and the residual:
    one half unit of the running sum of absolute values each."""
    M, k = ids.shape
    E, D = down.shape[:2]
    F = H.shape[1]
    out = np.zeros((M, D))
    T = np.zeros((M, D))
    for e in range(E):
        ps = np.nonzero(ids.reshape(-1) == e)[0]
        if ps.size:
            P, Tp = product(np.ascontiguousarray(H[ps]), down[e])
            g = wts.reshape(-1)[ps].astype(np.float64)[:, None]
            np.add.at(out, ps // k, g * P)
            np.add.at(T, ps // k, np.abs(g) * Tp)
    err = (BAR + (k * (F // 256) + 20) * lo.EPS) * T
    if residual is not None:
        out = out + residual
        err = err + lo.EPS * (np.abs(out) + err)
    return out, err


def assert_close(got, want, err, what=""):
    got = np.asarray(got, np.float64)
    assert got.shape == want.shape, (got.shape, want.shape)
    off = np.abs(got - want)
    bad = ~(off <= err)
    if bad.any():
        at = np.argwhere(bad)[:5].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside the bound, first {at}: "
                             f"{got[bad][:5]} against {want[bad][:5]}, allowed {err[bad][:5]}")
