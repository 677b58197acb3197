"""The layer oracle against hand-derived values and elementary identities (CPU only)."""
import math

import numpy as np
import pytest

from oracle import layer_oracle as lo


def test_activations_at_known_points():
    # silu(1) = 1/(1 + e^-1); gelu(1) = Phi(1); gelu_tanh(1) by its definition
    assert lo.act(1.0, "silu") == pytest.approx(1 / (1 + math.exp(-1)), rel=1e-15)
    assert lo.act(1.0, "gelu") == pytest.approx(0.8413447460685429, rel=1e-15)
    t = math.tanh(math.sqrt(2 / math.pi) * 1.044715)
    assert lo.act(1.0, "gelu_tanh") == pytest.approx(0.5 * (1 + t), rel=1e-15)
    for name in lo.ACTS:
        assert lo.act(0.0, name) == 0.0
    assert lo.act(-2.0, "relu") == 0.0 and np.isnan(lo.act(np.nan, "relu"))
    assert lo.act(-1e5, "silu") == 0.0 and lo.act(1e5, "gelu_tanh") == 1e5


@pytest.mark.parametrize("name", lo.ACTS)
def test_slopes_bound_the_activations(name):
    v = np.linspace(-12, 12, 200001)
    a = lo.act(v, name)
    assert np.max(np.abs(np.diff(a)) / np.diff(v)) <= lo.SLOPE[name]


def test_float32_activations_stay_inside_their_bound():
    """The kernels' formulas, evaluated in numpy float32, against the bound the tests use."""
    v = np.linspace(-30, 30, 20001).astype(np.float32)
    one = np.float32(1)

    def times_sigmoid(u):
        e = np.exp2(np.abs(u) * np.float32(-1.44269504))
        r = one / (one + e)
        return v * np.where(u >= 0, r, e * r)

    u2 = v * ((v * v) * np.float32(0.071354816) + np.float32(1.5957691216))
    t = np.abs(v)
    s = one / (one + np.float32(0.375) * t)
    p = np.zeros_like(s)
    for c in (-0.032911047, 0.13687992, -0.18652119, 0.050632391, 0.015627913, 0.088638239,
              0.12844568, 0.14960459, 0.14960338):
        p = p * s + np.float32(c)
    q = np.exp2(t * t * np.float32(-0.72134752)) * (p * s)
    gelu = v * np.where(v >= 0, one - q, q)
    for name, got in (("silu", times_sigmoid(v)), ("gelu_tanh", times_sigmoid(u2)), ("gelu", gelu)):
        assert got.dtype == np.float32
        off = np.abs(got.astype(np.float64) - lo.act(v, name))
        assert np.all(off <= lo.act_err(v.astype(np.float64), 0.0, name)), name


def test_route_by_hand():
    nan, inf = np.nan, np.inf
    logits = np.array([[0.0, 2.0, 2.0, -1.0],       # a tie: the lower expert first
                       [-inf, nan, 1.0, -inf],      # one that can be chosen
                       [-inf] * 4,                  # none
                       [inf, 0.0, inf, 1.0]])       # two share the softmax
    ids, w = lo.route(logits, 2, "softmax", True)
    assert ids.tolist() == [[1, 2], [2, -1], [-1, -1], [0, 2]]
    assert w.tolist() == [[0.5, 0.5], [1.0, 0.0], [0.0, 0.0], [0.5, 0.5]]
    _, w = lo.route(logits[:1], 2, "softmax", False)
    total = 2 + math.exp(-2) + math.exp(-3)
    np.testing.assert_allclose(w, [[1 / total, 1 / total]], rtol=1e-15)
    _, w = lo.route(np.array([[0.0, math.log(3.0)]]), 2, "sigmoid", False)
    np.testing.assert_allclose(w, [[0.75, 0.5]], rtol=1e-15)
    _, w = lo.route(np.array([[0.0, math.log(3.0)]]), 2, "sigmoid", True)
    np.testing.assert_allclose(w, [[0.6, 0.4]], rtol=1e-15)


def test_plan_by_hand():
    ids = np.array([[2, 0], [2, -1], [7, 2]])       # 7 is outside E = 4; expert 2 three times
    assert lo.plan(ids, 4).tolist() == [2, 4, 0, 0,
                                        0, 1 - 1, 1, 0, 2, 1, 3, 0, -1, 0, 0, 0, -1, 0, 0, 0,
                                        1, 0, 2, 5, -1, -1]


def test_epilogue_and_gated_by_hand():
    P, T = np.array([[1.0, -3.0]]), np.array([[2.0, 4.0]])
    out, err = lo.epilogue(P, T, 1e-5, "relu", bias=np.array([1.0, 1.0]),
                           residual=np.array([[10.0, 20.0]]))
    assert out.tolist() == [[12.0, 20.0]]
    assert np.all(err >= 1e-5 * T) and np.all(err < 1e-4)
    out, _ = lo.gated(P, T, 2 * P, T, 1e-5, "none")
    assert out.tolist() == [[2.0, 18.0]]
