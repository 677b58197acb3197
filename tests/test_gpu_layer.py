"""The layer operators on the GPU: the product's epilogue, the gated product, the router with its
plan, the experts' products and the whole layer, against the float64 oracle and, where the
arithmetic is the same, bit for bit against the plain product followed by float32 torch operations.
"""
import functools

import numpy as np
import pytest

import synth
from oracle import layer_oracle as lo
from tests import layer_util as lu
from tests.gpu_util import gpu_quantize, gpu_repack, say, to_dev

pytestmark = pytest.mark.gpu

mmq = pytest.importorskip("q4_q8_int8_amd")
torch = pytest.importorskip("torch")

NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "the gpu tests need a GPU"
    yield
    torch.cuda.synchronize()


def f32(*shape):
    return torch.full(shape, NAN, dtype=torch.float32, device="cuda")


def raw(n):
    return torch.zeros(max(n, 16), dtype=torch.uint8, device="cuda")


def host(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


# ---------------------------------------------------------------- the epilogue

# every kernel: the decode tile's forms (vector ALU 1, 2, 4 tokens, also with K over one step;
# matrix unit with 16, 8 and 4 wavefronts), skinny in both forms, the four template tiles, ragged
# rows and columns
EPI_SHAPES = [(1, 160, 512, 0), (1, 33, 4352, 0), (2, 64, 256, 0), (3, 100, 768, 0),
              (5, 160, 1024, 0), (16, 4100, 256, 0), (7, 8208, 256, 0), (9, 5120, 256, 0),
              (33, 70, 2048, mmq.MMQ_TILE_SKINNY), (64, 8192, 2048, mmq.MMQ_TILE_SKINNY),
              (40, 72, 512, mmq.MMQ_TILE_SMALL), (70, 258, 512, mmq.MMQ_TILE_MEDIUM),
              (70, 260, 512, mmq.MMQ_TILE_HALF), (130, 291, 512, mmq.MMQ_TILE_LARGE)]


@pytest.mark.parametrize("M,N,K,tile", EPI_SHAPES)
def test_epilogue_every_kernel(M, N, K, tile):
    """bias + residual without an activation is bit for bit the product plus two float32 sums; with
    an activation it is within the oracle's bound."""
    x = synth.activations("normal_outliers", M, K, 11 + M)
    w = lu.weights(N, K, 12 + N)
    rng = np.random.default_rng(M * N)
    b = rng.standard_normal(N).astype(np.float32)
    r = rng.standard_normal((M, N)).astype(np.float32)
    q8, rep, bias, res = gpu_quantize(x), gpu_repack(w, N, K), to_dev(b), to_dev(r)
    say("epilogue", (M, N, K), "tile", tile)
    plain, C = f32(M, N), f32(M, N)
    mmq.mmq_q4K_q8_1_ex(M, N, K, q8, rep, plain, force_tile=tile)
    info = mmq.mmq_last_kernel()
    mmq.mmq_q4K_q8_1_epilogue(M, N, K, q8, rep, C, force_tile=tile)
    assert mmq.mmq_last_kernel() == info
    assert np.array_equal(host(C), host(plain)), "an empty epilogue changes the product"
    mmq.mmq_q4K_q8_1_epilogue(M, N, K, q8, rep, C, bias=bias, residual=res, force_tile=tile)
    assert np.array_equal(host(C), host((plain + bias) + res))
    P, T = lu.product(x, w)
    for act in ("relu", "silu", "gelu", "gelu_tanh"):
        mmq.mmq_q4K_q8_1_epilogue(M, N, K, q8, rep, C.fill_(NAN), bias=bias,
                                  act=mmq.ACTIVATIONS[act], force_tile=tile)
        lu.assert_close(host(C), *lo.epilogue(P, T, lu.BAR, act, bias=b), what=act)
    C.copy_(res)                                   # the residual stream, updated in place
    mmq.mmq_q4K_q8_1_epilogue(M, N, K, q8, rep, C, residual=C, force_tile=tile)
    assert np.array_equal(host(C), host(plain + res))


@pytest.mark.parametrize("N", [320, 130])
def test_epilogue_with_split_k(N):
    M, K = 200, 2048
    x, w = synth.activations("normal", M, K, 5), lu.weights(N, K, 6)
    rng = np.random.default_rng(7)
    b, r = rng.standard_normal(N).astype(np.float32), rng.standard_normal((M, N)).astype(np.float32)
    q8, rep, bias, res = gpu_quantize(x), gpu_repack(w, N, K), to_dev(b), to_dev(r)
    ws = raw(4 * M * N * 4)
    how = dict(workspace=ws, splits=4, force_tile=mmq.MMQ_TILE_MEDIUM)
    say("epilogue split-K", (M, N, K))
    plain, C = f32(M, N), f32(M, N)
    mmq.mmq_q4K_q8_1_ex(M, N, K, q8, rep, plain, **how)
    mmq.mmq_q4K_q8_1_epilogue(M, N, K, q8, rep, C, bias=bias, residual=res, **how)
    assert mmq.mmq_last_kernel()["splits"] == 4
    assert np.array_equal(host(C), host((plain + bias) + res))
    mmq.mmq_q4K_q8_1_epilogue(M, N, K, q8, rep, C, bias=bias, act=mmq.MMQ_ACT_SILU, **how)
    P, T = lu.product(x, w)
    lu.assert_close(host(C), *lo.epilogue(P, T, lu.BAR, "silu", bias=b))


@pytest.mark.parametrize("M,N,K", [(1, 160, 512), (1, 40, 4352), (2, 100, 512), (4, 64, 256),
                                   (7, 33, 512), (20, 70, 512), (128, 64, 256)])
def test_epilogue_from_f32(M, N, K):
    x, w = synth.activations("normal_outliers", M, K, 21), lu.weights(N, K, 22)
    rng = np.random.default_rng(23)
    b, r = rng.standard_normal(N).astype(np.float32), rng.standard_normal((M, N)).astype(np.float32)
    xd, rep, bias, res = to_dev(x), gpu_repack(w, N, K), to_dev(b), to_dev(r)
    say("epilogue f32", (M, N, K))
    plain, C = f32(M, N), f32(M, N)
    mmq.mmq_q4K_f32(M, N, K, xd, rep, plain)
    mmq.mmq_q4K_f32_epilogue(M, N, K, xd, rep, C, bias=bias, residual=res)
    assert np.array_equal(host(C), host((plain + bias) + res))
    mmq.mmq_q4K_f32_epilogue(M, N, K, xd, rep, C, residual=res, act=mmq.MMQ_ACT_GELU)
    P, T = lu.product(x, w)
    lu.assert_close(host(C), *lo.epilogue(P, T, lu.BAR, "gelu", residual=r))


def test_activations_at_the_ends():
    """Sums that are huge, zero, infinite and NaN through the bias, against torch's float64
    activations: silu and gelu of -huge are 0, of +huge the value, of NaN NaN."""
    M, N, K = 1, 64, 256
    x, w = np.zeros((M, K), np.float32), lu.weights(N, K, 1)
    vals = np.array([0.0, -0.0, 1e-30, 88.0, -88.0, -89.0, -104.0, 1e4, -1e4, 3e38, -3e38, np.inf,
                     np.nan, -1e-42], np.float32)
    b = np.resize(vals, N)
    xd, rep, bias, C = to_dev(x), gpu_repack(w, N, K), to_dev(b), f32(M, N)
    z = torch.from_numpy(b.astype(np.float64))
    for act, ref in (("relu", torch.relu(z)), ("silu", torch.nn.functional.silu(z)),
                     ("gelu", torch.nn.functional.gelu(z)),
                     ("gelu_tanh", torch.nn.functional.gelu(z, approximate="tanh"))):
        mmq.mmq_q4K_f32_epilogue(M, N, K, xd, rep, C, bias=bias, act=mmq.ACTIVATIONS[act])
        got, want = host(C)[0].astype(np.float64), ref.numpy()
        assert np.array_equal(np.isnan(got), np.isnan(want)), act
        # 2^-20 relative; and where e^v is below 2^-126 (v < -87.34) it is taken as 0, for a result
        # of at most 87.34 * 2^-126 = 1.03e-36
        with np.errstate(invalid="ignore"):
            ok = np.isnan(want) | (got == want) | (np.abs(got - want) <= 2.0 ** -20 * np.abs(want)
                                                   + 1.1e-36)
        assert ok.all(), (act, b[~ok], got[~ok], want[~ok])


def test_activations_over_their_range():
    """Every activation at 4096 values of the sum, fed through the bias (the product is 0): errors
    against float64 within 2^-21 of max(|v|, 1), eight half units: the exponential and reciprocal, one
    unit each, the roundings of argument, sum and products, and gelu's fit of 2.3e-7 of a tail whose
    product with v is at most 0.17."""
    M, N, K = 1, 4096, 256
    v = np.concatenate([np.linspace(-20, 20, 2048), np.random.default_rng(0).standard_normal(1024),
                        np.geomspace(1e-6, 10, 512), -np.geomspace(1e-6, 10, 512)])
    v = v.astype(np.float32)
    w = lu.weights(N, K, 1)
    C, bias, rep = f32(M, N), to_dev(v), gpu_repack(w, N, K)
    x = torch.zeros(M, K, device="cuda")
    for act in ("silu", "gelu", "gelu_tanh"):
        mmq.mmq_q4K_f32_epilogue(M, N, K, x, rep, C, bias=bias, act=mmq.ACTIVATIONS[act])
        want = lo.act(v.astype(np.float64), act)
        lu.assert_close(host(C)[0], want, 2.0 ** -21 * np.maximum(np.abs(v), 1.0), what=act)
        # and relative to the value itself near 0, where it is v / 2
        near = np.abs(v) < 0.1
        assert np.all(np.abs(host(C)[0] - want)[near] <= 2.0 ** -20 * np.abs(want)[near]), act


# ---------------------------------------------------------------- the gated product

def pair(gate, up, F, K):
    rep = raw(mmq.mmq_q4K_pair_bytes(F, K)).fill_(0xA5)
    mmq.repack_q4_K_pair(to_dev(gate), to_dev(up), F, K, rep)
    return rep


@pytest.mark.parametrize("F,K", [(16, 256), (1, 512), (40, 256), (57, 768)])
def test_repack_pair_is_the_repack_of_the_packed_rows(F, K):
    gate, up = lu.weights(F, K, 1), lu.weights(F, K, 2)
    rows = 32 * ((F + 15) // 16)
    packed = np.zeros((rows, K // 256, 144), np.uint8)
    g, u = lu.pair_columns(F)
    packed[g], packed[u] = gate, up
    assert np.array_equal(host(pair(gate, up, F, K)), host(gpu_repack(packed, rows, K)))


GATED_SHAPES = [(1, 80, 512, 0), (1, 11, 4352, 0), (2, 40, 256, 0), (4, 33, 512, 0),
                (6, 70, 512, 0), (16, 2056, 256, 0), (9, 2500, 256, 0), (11, 4100, 256, 0),
                (33, 35, 2048, mmq.MMQ_TILE_SKINNY), (64, 4096, 2048, mmq.MMQ_TILE_SKINNY),
                (40, 36, 512, mmq.MMQ_TILE_SMALL), (70, 130, 512, mmq.MMQ_TILE_MEDIUM),
                (70, 132, 512, mmq.MMQ_TILE_HALF), (130, 147, 512, mmq.MMQ_TILE_LARGE)]


@pytest.mark.parametrize("M,F,K,tile", GATED_SHAPES)
def test_gated_every_kernel(M, F, K, tile):
    """The bilinear form is bit for bit the product over the packed rows, gate columns times up
    columns; the activations are within the oracle's bound."""
    x = synth.activations("normal_outliers", M, K, 31 + M)
    gate, up = lu.weights(F, K, 32), lu.weights(F, K, 33)
    q8, rep = gpu_quantize(x), pair(gate, up, F, K)
    rows = 32 * ((F + 15) // 16)
    say("gated", (M, F, K), "tile", tile)
    both, H = f32(M, rows), f32(M, F)
    mmq.mmq_q4K_q8_1_ex(M, rows, K, q8, rep, both, force_tile=tile)
    info = mmq.mmq_last_kernel()
    mmq.mmq_q4K_q8_1_gated(M, F, K, q8, rep, H, act=mmq.MMQ_ACT_NONE, force_tile=tile)
    assert mmq.mmq_last_kernel() == info
    g, u = (torch.from_numpy(c).cuda() for c in lu.pair_columns(F))
    assert np.array_equal(host(H), host(both[:, g] * both[:, u]))
    (G, TG), (U, TU) = lu.product(x, gate), lu.product(x, up)
    for act in ("silu", "gelu_tanh"):
        mmq.mmq_q4K_q8_1_gated(M, F, K, q8, rep, H.fill_(NAN), act=mmq.ACTIVATIONS[act],
                               force_tile=tile)
        lu.assert_close(host(H), *lo.gated(G, TG, U, TU, lu.BAR, act), what=act)


@pytest.mark.parametrize("F", [160, 67])
def test_gated_with_split_k(F):
    M, K = 200, 2048
    x, gate, up = synth.activations("normal", M, K, 5), lu.weights(F, K, 6), lu.weights(F, K, 7)
    q8, rep = gpu_quantize(x), pair(gate, up, F, K)
    rows = 32 * ((F + 15) // 16)
    how = dict(workspace=raw(3 * M * rows * 4), splits=3, force_tile=mmq.MMQ_TILE_SMALL)
    both, H = f32(M, rows), f32(M, F)
    say("gated split-K", (M, F, K))
    mmq.mmq_q4K_q8_1_ex(M, rows, K, q8, rep, both, **how)
    mmq.mmq_q4K_q8_1_gated(M, F, K, q8, rep, H, act=mmq.MMQ_ACT_NONE, **how)
    assert mmq.mmq_last_kernel()["splits"] == 3
    g, u = (torch.from_numpy(c).cuda() for c in lu.pair_columns(F))
    assert np.array_equal(host(H), host(both[:, g] * both[:, u]))


@pytest.mark.parametrize("M,F,K", [(1, 80, 512), (1, 20, 4352), (2, 50, 512), (4, 32, 256),
                                   (7, 17, 512), (20, 35, 512), (128, 32, 256)])
def test_gated_from_f32(M, F, K):
    x, gate, up = (synth.activations("normal_outliers", M, K, 41), lu.weights(F, K, 42),
                   lu.weights(F, K, 43))
    rep, H, rows = pair(gate, up, F, K), f32(M, F), 32 * ((F + 15) // 16)
    both = f32(M, rows)
    say("gated f32", (M, F, K))
    mmq.mmq_q4K_f32(M, rows, K, to_dev(x), rep, both)
    mmq.mmq_q4K_f32_gated(M, F, K, to_dev(x), rep, H, act=mmq.MMQ_ACT_NONE)
    g, u = (torch.from_numpy(c).cuda() for c in lu.pair_columns(F))
    assert np.array_equal(host(H), host(both[:, g] * both[:, u]))
    mmq.mmq_q4K_f32_gated(M, F, K, to_dev(x), rep, H)
    (G, TG), (U, TU) = lu.product(x, gate), lu.product(x, up)
    lu.assert_close(host(H), *lo.gated(G, TG, U, TU, lu.BAR, "silu"))


# ---------------------------------------------------------------- the router and the plan

def gpu_route(logits, k, score, renorm, planned):
    M, E = logits.shape
    ids = torch.full((M, k), -7, dtype=torch.int32, device="cuda")
    w = f32(M, k)
    plan = (torch.full((mmq.mmq_moe_plan_bytes(M, E, k) // 4,), -9, dtype=torch.int32,
                       device="cuda") if planned else None)
    mmq.mmq_moe_route(M, E, k, to_dev(logits), ids, w, plan, score=mmq.SCORES[score],
                      renorm=renorm)
    return ids, w, plan


def check_weights(got, want):
    """Relative 2^-17: an exponential's argument below 100 is rounded to half a unit, 100 * 2^-24,
    and the exponential, the sums of up to 512 values over lanes and registers (14 additions) and
    the quotient add less than 28 half units. Weights below float32's normal range: absolute."""
    assert np.all(np.abs(got - want) <= 2.0 ** -17 * want + 1.2e-38), (got, want)


@pytest.mark.parametrize("M,E,k", [(1, 8, 2), (1, 64, 8), (64, 64, 8), (5, 1, 1), (3, 63, 63),
                                   (2, 65, 5), (17, 128, 6), (9, 200, 8), (64, 256, 8),
                                   (7, 512, 64), (8, 500, 10)])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False),
                                          ("sigmoid", True), ("sigmoid", False)])
def test_route(M, E, k, score, renorm):
    rng = np.random.default_rng(M * 1000 + E)
    logits = (3 * rng.standard_normal((M, E))).astype(np.float32)
    logits[M // 2] = np.round(logits[M // 2])                 # ties
    say("route", (M, E, k), score, renorm)
    ids, w, plan = gpu_route(logits, k, score, renorm, True)
    want, ww = lo.route(logits, k, score, renorm)
    assert np.array_equal(host(ids), want)
    check_weights(host(w), ww)
    assert np.array_equal(host(plan), lo.plan(want, E))
    ids2, w2, _ = gpu_route(logits, k, score, renorm, False)
    assert np.array_equal(host(ids2), want) and np.array_equal(host(w2), host(w))


def test_route_masked_and_extreme_rows():
    inf, nan, big = np.inf, np.nan, np.finfo(np.float32).max
    E, k = 70, 4
    logits = np.random.default_rng(1).standard_normal((12, E)).astype(np.float32)
    logits[0] = -inf                                  # nothing left
    logits[1] = nan
    logits[2, 3:] = -inf                              # fewer than k
    logits[3, ::2] = nan
    logits[4] = -big                                  # the type's lowest value: a tie of 70
    logits[5, [69, 4]] = inf
    logits[6] = 0.0
    logits[6, 1::2] = -0.0                            # equal to 0
    logits[7] = big
    logits[8] = -200.0                                # every sigmoid 0 in float32
    logits[9, 5], logits[9, 6] = 1e-42, -1e-42        # denormals are ordered
    logits[9, 7:], logits[9, :5] = -1.0, -1.0
    logits[10] = -inf
    logits[10, 66] = -big
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            say("route extremes", score, renorm)
            with np.errstate(over="ignore"):
                want, ww = lo.route(logits, k, score, renorm)
            ids, w, plan = gpu_route(logits, k, score, renorm, True)
            assert np.array_equal(host(ids), want), score
            got = host(w)
            if score == "sigmoid" and renorm:
                # 1 / (1 + e^200) is 0 in float32: the sum is 0 and so are the weights
                assert np.all(got[8] == 0)
                ww[8] = 0
                for r in (4, 10):
                    assert np.all(got[r] == 0)
                    ww[r] = 0
            check_weights(got, ww)
            assert np.array_equal(host(plan), lo.plan(want, E))


def test_route_sigmoid_weights_of_very_negative_logits():
    """Normalised sigmoid weights go by the ratios of the scores, also where e^-l is past float32's
    range (l < -88.7); they are 0 only where the greatest chosen score itself is 0 in float32 (l below
    -150 ln 2 = -103.97). The tolerance is check_weights', whose argument below 100 covers the
    differences of logits that give a normal weight (87.3)."""
    inf, k = np.inf, 4
    rows = [[-88.0, -89.0, -90.0], [-89.0, -89.5], [-100.0, -101.0, -103.0, -103.9],
            [-103.9] * 6, [-103.97, -104.5, -150.0, -300.0], [-103.98, -103.99],
            [-103.97208], [-103.972084], [-200.0] * 4,
            [-20.0, -88.8, -95.0, -107.0], [-17.0, -16.0, -18.5, -17.5], [5.0, -50.0, -87.0, -100.0],
            [0.0, -80.0, -87.0], [-0.5, -88.0, -87.5], [inf, -88.0, -90.0], [-inf], [-95.0],
            [40.0, 20.0, -60.0], [-30.0, -30.0, -118.0]]
    for E in (8, 70, 130):
        logits = np.full((len(rows), E), -inf, np.float32)
        for t, r in enumerate(rows):
            logits[t, E - len(r):] = r
        want, _ = lo.route(logits, k, "sigmoid", False)
        z = np.take_along_axis(logits.astype(np.float64), np.maximum(want, 0), 1)
        s = np.where(want >= 0, 1.0 / (1.0 + np.exp(-z)), 0.0)
        top = s[:, 0].astype(np.float32)               # correctly rounded: 0 below 2^-150
        total = np.where(top > 0, s.sum(1), 1.0)
        w = np.where(top[:, None] > 0, s / total[:, None], 0.0)
        say("route: very negative logits", E)
        ids, got, _ = gpu_route(logits, k, "sigmoid", True, True)
        assert np.array_equal(host(ids), want)
        check_weights(host(got), w)
        _, got, _ = gpu_route(logits, k, "sigmoid", False, False)
        check_weights(host(got), s)


def test_route_many_tokens():
    M, E, k = 4099, 96, 6
    logits = np.random.default_rng(3).standard_normal((M, E)).astype(np.float32)
    ids, w, _ = gpu_route(logits, k, "softmax", True, False)
    z = torch.from_numpy(logits).double()
    order = torch.sort(z, dim=1, descending=True, stable=True)
    assert np.array_equal(host(ids), order.indices[:, :k].numpy().astype(np.int32))
    check_weights(host(w), torch.softmax(order.values[:, :k], 1).numpy())


@pytest.mark.parametrize("M,E,k", [(1, 4, 2), (64, 512, 8), (64, 3, 3), (8, 64, 64), (33, 17, 4)])
def test_plan_from_ids(M, E, k):
    rng = np.random.default_rng(E)
    cases = [rng.integers(0, E, (M, k)),              # a token may name an expert twice
             rng.integers(-2, E + 3, (M, k)),         # some name none
             np.full((M, k), -1), np.full((M, k), E - 1), np.full((M, k), 2 ** 31 - 1)]
    for ids in cases:
        ids = ids.astype(np.int32)
        plan = torch.full((mmq.mmq_moe_plan_bytes(M, E, k) // 4,), 77, dtype=torch.int32,
                          device="cuda")
        say("plan", (M, E, k))
        mmq.mmq_moe_plan(M, E, k, to_dev(ids), plan)
        assert np.array_equal(host(plan), lo.plan(ids, E))


# ---------------------------------------------------------------- the experts' products

class Experts:
    def __init__(self, E, D, F, seed=50):
        self.E, self.D, self.F = E, D, F
        self.gate = np.stack([lu.weights(F, D, seed + 3 * e) for e in range(E)])
        self.up = np.stack([lu.weights(F, D, seed + 3 * e + 1) for e in range(E)])
        self.down = (np.stack([lu.weights(D, F, seed + 3 * e + 2) for e in range(E)])
                     if F % 256 == 0 else None)
        self.w_in = torch.cat([pair(self.gate[e], self.up[e], F, D) for e in range(E)])
        if self.down is not None:
            self.w_out = torch.cat([gpu_repack(self.down[e], D, F) for e in range(E)])


def ids_of(kind, M, E, k, seed=0):
    rng = np.random.default_rng(seed)
    if kind == "distinct":
        ids = np.stack([rng.permutation(E)[:k] for _ in range(M)])
    elif kind == "repeated":                          # any expert, also twice in a token
        ids = rng.integers(0, E, (M, k))
    elif kind == "one":                               # everything to one expert
        ids = np.full((M, k), E - 1)
    elif kind == "padded":                            # whole tokens and single slots without
        ids = np.stack([rng.permutation(E)[:k] for _ in range(M)])
        ids[M // 2:, :] = -1
        ids[0, k - 1] = E + 5
    elif kind == "none":
        ids = np.full((M, k), -1)
    return ids.astype(np.int32)


def plan_of(ids, E):
    M, k = ids.shape
    plan = torch.empty(mmq.mmq_moe_plan_bytes(M, E, k) // 4, dtype=torch.int32, device="cuda")
    mmq.mmq_moe_plan(M, E, k, to_dev(ids), plan)
    return plan


def gpu_gated(ex, x, ids, act="silu"):
    M, k = ids.shape
    H = f32(M * k, ex.F)
    mmq.mmq_q4K_moe_gated(M, ex.E, k, ex.F, ex.D, to_dev(x), plan_of(ids, ex.E), ex.w_in, H,
                          raw(mmq.mmq_q8_1_bytes(M, ex.D)).fill_(0xFF),
                          act=mmq.ACTIVATIONS[act])
    return H


def gpu_down(ex, H, ids, wts, residual=None, out=None):
    M, k = ids.shape
    out = f32(M, ex.D) if out is None else out
    mmq.mmq_q4K_moe_down(M, ex.E, k, ex.D, ex.F, to_dev(H), plan_of(ids, ex.E), to_dev(wts),
                         ex.w_out, out, raw(mmq.mmq_q8_1_bytes(M * k, ex.F)).fill_(0xFF),
                         residual=residual)
    return out


MOE = [(1, 8, 2, 512, 256), (1, 16, 8, 2048, 512), (2, 4, 4, 256, 768), (3, 8, 3, 768, 40),
       (4, 8, 2, 512, 33), (5, 8, 4, 512, 256), (16, 4, 2, 256, 512), (17, 3, 3, 512, 256),
       (64, 8, 2, 256, 256), (64, 12, 8, 256, 256), (3, 16, 2, 2048, 64), (6, 3, 2, 4352, 24),
       (9, 3, 3, 512, 768)]


@pytest.mark.parametrize("M,E,k,D,F", MOE)
@pytest.mark.parametrize("kind", ["distinct", "repeated", "one", "padded", "none"])
def test_moe_gated(M, E, k, D, F, kind):
    ex = Experts(E, D, F)
    x, ids = synth.activations("normal_outliers", M, D, 60 + M), ids_of(kind, M, E, k)
    say("moe gated", (M, E, k, D, F), kind)
    got = host(gpu_gated(ex, x, ids))
    want, err = lu.experts_gated(x, ids, ex.gate, ex.up, "silu")
    none = np.isnan(want).all(axis=1)
    assert np.all(np.isnan(got[none])), "a row without an expert was written"
    lu.assert_close(got[~none], want[~none], err[~none])


@pytest.mark.parametrize("M,E,k,D,F", [c for c in MOE if c[4] % 256 == 0]
                         + [(1, 4, 2, 20, 512), (6, 4, 2, 45, 512), (1, 3, 2, 2064, 768),
                            (2, 3, 2, 2064, 256), (12, 3, 2, 2070, 512)])
@pytest.mark.parametrize("kind", ["distinct", "repeated", "one", "padded", "none"])
def test_moe_down(M, E, k, D, F, kind):
    ex = ExpertsDown(E, D, F)
    rng = np.random.default_rng(M + D)
    H = synth.activations("swiglu", M * k, F, 70 + M)
    ids = ids_of(kind, M, E, k)
    H[~((ids >= 0) & (ids < E)).reshape(-1)] = np.nan     # rows that nobody uses
    wts = rng.random((M, k)).astype(np.float32)
    wts[~((ids >= 0) & (ids < E))] = np.nan
    res = rng.standard_normal((M, D)).astype(np.float32)
    say("moe down", (M, E, k, D, F), kind)
    clean = np.nan_to_num(H)
    for r in (None, res):
        got = host(gpu_down(ex, H, ids, wts, None if r is None else to_dev(r)))
        lu.assert_close(got, *lu.experts_down(clean, ids, np.nan_to_num(wts), ex.down, r))
    inplace = to_dev(res)
    gpu_down(ex, H, ids, wts, inplace, out=inplace)
    assert np.array_equal(host(inplace), got)


class ExpertsDown:
    def __init__(self, E, D, F, seed=50):
        self.E, self.D, self.F = E, D, F
        self.down = np.stack([lu.weights(D, F, seed + e) for e in range(E)])
        self.w_out = torch.cat([gpu_repack(self.down[e], D, F) for e in range(E)])


# ---------------------------------------------------------------- more than one step of K a wavefront

# every form of the down product, its wavefronts walking 2 to 17 steps of their part of K, with an odd
# number of super-blocks (so that the last step is partly empty) and with several groups of columns
DOWN_STEPS = [(1, 8, 2, 512, 4352),     # vector ALU, 8 rows, one token: 5 steps in 4 parts
              (1, 16, 16, 72, 2304),    # ... 3 steps, one part
              (1, 6, 3, 2064, 4352),    # 16 rows, one token: 9 steps in 4 parts
              (4, 12, 2, 512, 4352),    # 8 rows, groups of 3 columns: 5 steps in 2 parts
              (8, 8, 2, 512, 4352),     # matrix unit, 8 rows, groups of 8: 9 steps in 2 parts
              (12, 16, 2, 40, 4352),    # 8 rows, groups of 3: 5 steps, one part, 16 experts
              (8, 8, 2, 2064, 4352),    # vector ALU, 16 rows, groups of 4: 9 steps in 2 parts
              (16, 3, 3, 2064, 2304),   # matrix unit, 16 rows, groups of 16: 9 steps in 4 parts
              (20, 2, 2, 2050, 4352)]   # ... 17 steps in 8 parts, an expert of 20 columns


@functools.lru_cache(maxsize=1)
def down_experts(E, D, F):
    return ExpertsDown(E, D, F)


@pytest.mark.parametrize("M,E,k,D,F", DOWN_STEPS)
@pytest.mark.parametrize("kind", ["distinct", "one", "padded"])
def test_moe_down_over_several_steps(M, E, k, D, F, kind):
    ex = down_experts(E, D, F)
    H = synth.activations("swiglu", M * k, F, 90 + M)
    ids = ids_of(kind, M, E, k)
    rng = np.random.default_rng(M + F)
    wts, res = rng.random((M, k)).astype(np.float32), rng.standard_normal((M, D)).astype(np.float32)
    say("moe down, several steps", (M, E, k, D, F), kind)
    got = host(gpu_down(ex, H, ids, wts, to_dev(res)))
    lu.assert_close(got, *lu.experts_down(H, ids, wts, ex.down, res))


# the gated product: one token (4 wavefronts over 9 or 5 steps; a token that names an expert three
# times walks K again for each), and the matrix unit with more than 16 columns (5 steps, 2 wavefronts)
GATED_STEPS = [(1, 8, 2, 4352, 40), (1, 4, 3, 2304, 33), (17, 2, 2, 1280, 40), (5, 8, 2, 2304, 24)]


@pytest.mark.parametrize("M,E,k,D,F", GATED_STEPS)
@pytest.mark.parametrize("kind", ["distinct", "repeated", "one", "padded"])
def test_moe_gated_over_several_steps(M, E, k, D, F, kind):
    ex = Experts(E, D, F)
    x, ids = synth.activations("normal_outliers", M, D, 95 + M), ids_of(kind, M, E, k)
    say("moe gated, several steps", (M, E, k, D, F), kind)
    got = host(gpu_gated(ex, x, ids))
    want, err = lu.experts_gated(x, ids, ex.gate, ex.up, "silu")
    none = np.isnan(want).all(axis=1)
    assert np.all(np.isnan(got[none])), "a row without an expert was written"
    lu.assert_close(got[~none], want[~none], err[~none])


def test_many_experts():
    """The plan's largest sizes: 512 experts, 512 pairs, all different and all the same."""
    M, E, k, D, F = 64, 512, 8, 256, 256
    ex = Experts(E, D, F)
    x = synth.activations("normal", M, D, 8)
    for ids in (np.arange(512).reshape(M, k).astype(np.int32), np.full((M, k), 511, np.int32)):
        H = host(gpu_gated(ex, x, ids))
        lu.assert_close(H, *lu.experts_gated(x, ids, ex.gate, ex.up, "silu"))
        wts = np.random.default_rng(9).random((M, k)).astype(np.float32)
        lu.assert_close(host(gpu_down(ex, H, ids, wts)),
                        *lu.experts_down(H, ids, wts, ex.down, None))


def test_expert_weights_past_4_gib():
    """The last of 512 experts starts 4.3 GB into the weights."""
    M, E, k, D, F = 2, 512, 2, 4096, 1840
    n = mmq.mmq_q4K_pair_bytes(F, D)
    assert (E - 1) * n > 2 ** 32
    w_in = torch.empty(E * n, dtype=torch.uint8, device="cuda")   # only two experts are written
    gate = {e: lu.weights(F, D, 2 * e) for e in (0, E - 1)}
    up = {e: lu.weights(F, D, 2 * e + 1) for e in (0, E - 1)}
    for e in gate:
        mmq.repack_q4_K_pair(to_dev(gate[e]), to_dev(up[e]), F, D, w_in[e * n:(e + 1) * n])
    x = synth.activations("normal", M, D, 3)
    ids = np.array([[0, E - 1], [E - 1, -1]], np.int32)
    H = f32(M * k, F)
    say("experts past 4 GiB")
    mmq.mmq_q4K_moe_gated(M, E, k, F, D, to_dev(x), plan_of(ids, E), w_in, H,
                          raw(mmq.mmq_q8_1_bytes(M, D)))
    got = host(H)
    for p, (t, e) in enumerate(((0, 0), (0, E - 1), (1, E - 1))):
        (G, TG), (U, TU) = lu.product(x[t:t + 1], gate[e]), lu.product(x[t:t + 1], up[e])
        want, err = lo.gated(G, TG, U, TU, lu.BAR, "silu")
        lu.assert_close(got[p:p + 1], want, err)


def test_moe_gated_one_expert_per_token_is_the_gated_product():
    """With one expert every pair is a row of the dense gated product, within both bounds."""
    M, D, F = 16, 1024, 256
    ex = Experts(1, D, F)
    x, ids = synth.activations("normal", M, D, 1), np.zeros((M, 1), np.int32)
    for act in mmq.ACTIVATIONS:
        got = host(gpu_gated(ex, x, ids, act))
        want, err = lu.experts_gated(x, ids, ex.gate, ex.up, act)
        lu.assert_close(got, want, err, what=act)


# ---------------------------------------------------------------- together

def layer(ex, x, logits, k, score, renorm, residual=None, stream=None):
    M = x.shape[0]
    out = f32(M, ex.D)
    ws = raw(mmq.mmq_moe_workspace_bytes(M, ex.E, k, ex.D, ex.F)).fill_(0xFF)
    mmq.mmq_q4K_moe(M, ex.E, k, ex.D, ex.F, x, logits, ex.w_in, ex.w_out, out, ws,
                    score=mmq.SCORES[score], renorm=renorm, residual=residual, stream=stream)
    return out, ws


@pytest.mark.parametrize("M,E,k,D,F", [(1, 16, 4, 512, 256), (4, 16, 4, 512, 512),
                                       (13, 8, 2, 256, 768), (64, 8, 2, 512, 256)])
def test_whole_layer_is_its_three_calls(M, E, k, D, F):
    ex = Experts(E, D, F)
    x = to_dev(synth.activations("normal_outliers", M, D, 3))
    logits = np.random.default_rng(4).standard_normal((M, E)).astype(np.float32)
    logits[M // 2] = -np.inf                          # a padded token
    res = to_dev(synth.activations("normal", M, D, 5))
    say("layer", (M, E, k, D, F))
    out, _ = layer(ex, x, to_dev(logits), k, "softmax", True, residual=res)
    ids, w, plan = gpu_route(logits, k, "softmax", True, True)
    H, want = f32(M * k, F), f32(M, D)
    mmq.mmq_q4K_moe_gated(M, E, k, F, D, x, plan, ex.w_in, H, raw(mmq.mmq_q8_1_bytes(M, D)))
    mmq.mmq_q4K_moe_down(M, E, k, D, F, H, plan, w, ex.w_out, want,
                         raw(mmq.mmq_q8_1_bytes(M * k, F)), residual=res)
    assert np.array_equal(host(out), host(want))
    assert np.array_equal(host(out)[M // 2], host(res)[M // 2])
    ids, w = host(ids), host(w)
    lu.assert_close(host(want), *lu.experts_down(np.nan_to_num(host(H)), ids, w, ex.down, host(res)))


@pytest.mark.parametrize("M", [1, 6])
def test_decoder_block_in_a_graph(M):
    """Output projection with the residual, gated feed-forward, down projection with the residual,
    then an expert layer, as a decoder runs them: captured, replayed over changed inputs, each
    replay against the eager calls."""
    D, F, E, k = 512, 768, 8, 2
    rep = gpu_repack(lu.weights(D, D, 1), D, D)
    ffn = pair(lu.weights(F, D, 2), lu.weights(F, D, 3), F, D)
    down = gpu_repack(lu.weights(D, F, 4), D, F)
    ex = Experts(E, D, F)
    x, a = f32(M, D), f32(M, D)
    logits = f32(M, E)
    y, H, z, out = f32(M, D), f32(M, F), f32(M, D), f32(M, D)
    q8 = raw(max(mmq.mmq_q8_1_bytes(M, D), mmq.mmq_q8_1_bytes(M, F)))
    ws = raw(mmq.mmq_moe_workspace_bytes(M, E, k, D, F))

    def step():
        mmq.quantize_q8_1(a, M, D, q8)
        mmq.mmq_q4K_q8_1_epilogue(M, D, D, q8, rep, y, residual=x)
        mmq.quantize_q8_1(y, M, D, q8)
        mmq.mmq_q4K_q8_1_gated(M, F, D, q8, ffn, H)
        mmq.mmq_q4K_f32_epilogue(M, D, F, H, down, z, residual=y)
        mmq.mmq_q4K_moe(M, E, k, D, F, z, logits, ex.w_in, ex.w_out, out, ws, residual=z)

    def inputs(seed):
        x.copy_(to_dev(synth.activations("normal_outliers", M, D, seed)))
        a.copy_(to_dev(synth.activations("normal", M, D, seed + 1)))
        logits.copy_(to_dev(np.random.default_rng(seed).standard_normal((M, E)).astype(np.float32)))

    wants = []
    for seed in (1, 2, 3):
        inputs(seed)
        step()
        wants.append(host(out).copy())
    assert np.isfinite(wants[0]).all() and not np.array_equal(wants[0], wants[1])
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    say("decoder block: capture", M)
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            step()
    torch.cuda.synchronize()
    for seed, want in zip((1, 2, 3), wants):
        inputs(seed)
        out.fill_(NAN)
        for t in (ws, q8):                            # eager work on the scratch in between
            t.fill_(0xFF)
        torch.cuda.synchronize()
        g.replay()
        assert np.array_equal(host(out), want), seed


def test_layer_on_two_streams_at_once():
    M, E, k, D, F = 3, 8, 2, 512, 256
    ex = Experts(E, D, F)
    runs = []
    for seed in (3, 4):
        x = to_dev(synth.activations("normal", M, D, seed))
        logits = to_dev(np.random.default_rng(seed).standard_normal((M, E)).astype(np.float32))
        want = host(layer(ex, x, logits, k, "sigmoid", True)[0])
        out, ws = f32(M, D), raw(mmq.mmq_moe_workspace_bytes(M, E, k, D, F))
        runs.append((x, logits, out, ws, want, torch.cuda.Stream()))
    torch.cuda.synchronize()
    say("layer on two streams", (M, E, k, D, F))
    for _ in range(20):                               # a workspace of its own for each stream
        for x, logits, out, ws, _, s in runs:
            mmq.mmq_q4K_moe(M, E, k, D, F, x, logits, ex.w_in, ex.w_out, out, ws,
                            score=mmq.SCORES["sigmoid"], stream=s)
    torch.cuda.synchronize()
    for _, _, out, _, want, _ in runs:
        assert np.array_equal(host(out), want)


def test_a_plan_of_nonsense_selects_nothing():
    """The products check what they read of a plan: entries outside its own sizes have no pairs."""
    M, E, k, D, F = 5, 8, 2, 512, 256
    ex = Experts(E, D, F)
    P, entries = M * k, min(E, M * k)
    x = to_dev(synth.activations("normal", M, D, 3))
    res, w = to_dev(synth.activations("normal", M, D, 4)), f32(M, k).fill_(1.0)
    bad = [(E, 0, 1), (-1, 0, 1), (0, P + 1, 0), (0, -1, 2), (0, 0, P + 1), (0, 0, -1),
           (0, P, 1), (1 << 30, 1 << 30, 1 << 30)]
    for used in (entries, entries + 1, -1, 1 << 30):
        plan = np.full(4 + 4 * entries + P, (1 << 31) - 1, np.int32)
        plan[0] = used
        for u in range(entries):
            plan[4 + 4 * u:7 + 4 * u] = bad[u % len(bad)]
        H, out = f32(P, F), f32(M, D)
        say("nonsense plan", used)
        mmq.mmq_q4K_moe_gated(M, E, k, F, D, x, to_dev(plan), ex.w_in, H,
                              raw(mmq.mmq_q8_1_bytes(M, D)))
        assert np.isnan(host(H)).all()
        mmq.mmq_q4K_moe_down(M, E, k, D, F, H.fill_(1.0), to_dev(plan), w, ex.w_out, out,
                             raw(mmq.mmq_q8_1_bytes(P, F)), residual=res)
        assert np.array_equal(host(out), host(res))


def test_results_repeat_bit_for_bit():
    M, E, k, D, F = 33, 8, 3, 512, 512
    ex = Experts(E, D, F)
    x, ids = synth.activations("normal", M, D, 1), ids_of("repeated", M, E, k)
    H = host(gpu_gated(ex, x, ids))
    wts = np.random.default_rng(2).random((M, k)).astype(np.float32)
    out = host(gpu_down(ex, H, ids, wts))
    for _ in range(3):
        assert np.array_equal(host(gpu_gated(ex, x, ids)), H)
        assert np.array_equal(host(gpu_down(ex, H, ids, wts)), out)


def test_python_checks_tensors():
    x = torch.zeros(2, 256, device="cuda")
    rep = raw(mmq.mmq_q4K_pair_bytes(16, 256))
    with pytest.raises(mmq.MMQArgumentError):
        mmq.mmq_q4K_f32_gated(2, 16, 256, x.double(), rep, f32(2, 16))
    with pytest.raises(mmq.MMQArgumentError):
        mmq.mmq_q4K_f32_gated(2, 16, 256, x, rep[:-16], f32(2, 16))
    with pytest.raises(mmq.MMQArgumentError):
        mmq.mmq_q4K_f32_gated(2, 16, 256, x, rep, f32(16, 2).t())
    with pytest.raises(mmq.MMQArgumentError):
        mmq.mmq_q4K_f32_epilogue(2, 16, 256, x, rep, f32(2, 16), bias=f32(15))
    with pytest.raises(mmq.MMQArgumentError):
        mmq.mmq_moe_route(2, 8, 2, f32(2, 8), torch.zeros(2, 2, dtype=torch.int64, device="cuda"),
                          f32(2, 2))
    with pytest.raises(mmq.MMQArgumentError):
        mmq.mmq_q4K_moe_down(2, 8, 2, 16, 256, f32(4, 256), torch.zeros(23, dtype=torch.int32,
                             device="cuda"), f32(2, 2), raw(8 * 4608), f32(2, 16), raw(1 << 16))


def test_current_device_and_stream_are_torch_s():
    """The binding asks torch's C module for the device and the stream: the same as torch.cuda's."""
    assert mmq._here() == torch.cuda.current_device()
    streams = [torch.cuda.default_stream(), torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        with torch.cuda.stream(s):
            assert mmq._stream(None) == torch.cuda.current_stream().cuda_stream == s.cuda_stream
            assert mmq._stream(None, mmq._here()) == s.cuda_stream
            assert mmq._stream(s) == s.cuda_stream
    assert mmq._stream(None) == torch.cuda.current_stream().cuda_stream
