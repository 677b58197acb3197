"""Oracle of the layer operators beside the product: its epilogue, the gated product, the router,
the experts' plan and their products. float64 numpy, from the definitions; integers exact.

Each product result comes with a bound scale T, the sum of the absolute values of its terms, and
the functions here carry both through the epilogue: `err` is how far a float32 result may be off
when the product itself is within `bar * T`, with half a unit in the last place (2^-24 of the
value) for every float32 rounding behind it.
"""
from __future__ import annotations

import math

import numpy as np

EPS = 2.0 ** -24

ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
# The greatest slope of each activation: relu and none 1; silu 1.0998; gelu 1.1290; gelu_tanh 1.1293.
SLOPE = {"none": 1.0, "relu": 1.0, "silu": 1.1, "gelu": 1.13, "gelu_tanh": 1.13}

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def act(v, name: str):
    """The activation in float64."""
    v = np.asarray(v, dtype=np.float64)
    if name == "none":
        return v
    if name == "relu":
        return np.where(v < 0, 0.0, v)
    if name == "gelu":
        return 0.5 * v * _erfc(-v / math.sqrt(2.0))
    if name == "silu":
        u = v
    elif name == "gelu_tanh":
        u = 2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)
    else:
        raise ValueError(name)
    # v / (1 + e^-u) without overflow
    e = np.exp(-np.abs(u))
    return v * np.where(u >= 0, 1.0, e) / (1.0 + e)


def act_err(z, dz, name: str):
    """Error of a float32 activation of z known to within dz: the slope carries dz; the up to
    three roundings of the exponential's (or erfc's) argument u reach the result as |z u s(1 - s)|,
    s = 1/(1 + e^-u), at most 1/2 half unit each, and are counted as 8 half units of max(|z|, 1)
    together; the exponential, the sum, the quotient and a product are within 16 half units of a
    result that is at most |z|."""
    if name in ("none", "relu"):
        return dz
    z = np.abs(z)
    return SLOPE[name] * dz + 8 * EPS * np.maximum(z, 1.0) + 16 * EPS * z


def epilogue(P, T, bar, name="none", bias=None, residual=None):
    """(act(P + bias) + residual, its error bound)."""
    z, dz = P, bar * T
    if bias is not None:
        z = P + np.asarray(bias, np.float64)
        dz = dz + EPS * (np.abs(z) + dz)
    out, err = act(z, name), act_err(z, dz, name)
    if residual is not None:
        out = out + np.asarray(residual, np.float64)
        err = err + EPS * (np.abs(out) + err)
    return out, err


def gated(G, TG, U, TU, bar, name):
    """(act(G) * U, its error bound)."""
    a, da = act(G, name), act_err(G, bar * TG, name)
    du = bar * TU
    out = a * U
    err = da * np.abs(U) + np.abs(a) * du + da * du
    return out, err + EPS * (np.abs(out) + err)


def route(logits, k: int, score: str, renorm: bool):
    """(ids int32 [M, k], weights float64 [M, k]): the k greatest logits of each row, equal ones in
    increasing order; -inf and NaN are never chosen (id -1, weight 0)."""
    logits = np.asarray(logits, np.float64)
    M, E = logits.shape
    ids = np.full((M, k), -1, np.int32)
    w = np.zeros((M, k))
    for t in range(M):
        can = [e for e in range(E) if logits[t, e] > -np.inf]
        chosen = sorted(can, key=lambda e: (-logits[t, e], e))[:k]
        if not chosen:
            continue
        v = logits[t, chosen]
        if score == "softmax":
            top = v[0]

            def below(x):
                less = x != top
                return np.where(less, np.exp(np.subtract(x, top, where=less, out=np.zeros(x.shape))),
                                1.0)
            s = below(v)
            total = s.sum() if renorm else below(logits[t, can]).sum()
            s = s / total
        else:
            s = 1.0 / (1.0 + np.exp(-v))
            if renorm:
                s = s / s.sum() if s.sum() > 0 else np.zeros_like(s)
        ids[t, :len(chosen)] = chosen
        w[t, :len(chosen)] = s
    return ids, w


def plan(ids, E: int):
    """The plan of ids [M, k] as int32: [used, pairs, 0, 0], entries [expert, first, pairs, 0] and
    the pairs sorted by expert."""
    flat = np.asarray(ids).reshape(-1)
    P = flat.size
    lists = [[p for p in range(P) if flat[p] == e] for e in range(E)]
    rows, order = [], []
    for e in range(E):
        if lists[e]:
            rows.append([e, len(order), len(lists[e]), 0])
            order += lists[e]
    used = len(rows)
    rows += [[-1, 0, 0, 0]] * (min(E, P) - used)
    head = [used, len(order), 0, 0]
    order += [-1] * (P - len(order))
    return np.array(head + [v for r in rows for v in r] + order, np.int32)


def groups(ids, E: int):
    """(offsets [E + 1], order, place) of ids [M, k], int32: where each expert's pairs begin, the pairs
    sorted by expert (those without one -1, at the end), and the place of each."""
    flat = np.asarray(ids).reshape(-1)
    P = flat.size
    offsets, order = [0], []
    for e in range(E):
        order += np.nonzero(flat == e)[0].tolist()
        offsets.append(len(order))
    place = np.full(P, -1, np.int32)
    place[order] = np.arange(len(order))
    order += [-1] * (P - len(order))
    return np.array(offsets, np.int32), np.array(order, np.int32), place
